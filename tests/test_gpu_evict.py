"""qsa_evict_select against a sort (cache_cases.keep_units): equal lists, no tolerance."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev, keep_units

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def call(qsa, mass, length, tokens, keep, first, last, unit, spare=3, stream=None):
    n = mass.shape[0]
    cols = min(tokens, keep + unit - 1) + spare
    sel = torch.full((n, cols), -5, dtype=torch.int32, device="cuda")
    n_sel = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    st = qsa.new_status()
    m, ln = dev(mass), dev(np.asarray(length, np.int32))
    torch.cuda.synchronize()
    qsa.qsa_evict_select(m, mass.shape[2], mass.shape[1], ln, n, tokens, keep, first, last, unit, sel, cols, n_sel, st,
                         stream=stream)
    torch.cuda.synchronize()
    return sel.cpu().numpy(), n_sel.cpu().numpy(), qsa.qsa_read_status(st)


def check(mass, length, keep, first, last, unit, sel, n_sel):
    for i, n in enumerate(length):
        want = keep_units(mass[i], int(n), keep, first, last, unit)
        assert n_sel[i] == len(want), i
        assert np.array_equal(sel[i, :len(want)], want), i
        assert np.all(sel[i, len(want):] == -5), "entries past the list were written"


def draws(rng, kind, shape):
    u = rng.random(shape, dtype=np.float32)
    if kind == "heavy":
        return (u ** 12).astype(np.float32)
    if kind == "ties":
        return (np.floor(u * 6) / 4).astype(np.float32)
    if kind == "zeros":
        x = np.where(u < 0.9, 0.0, u).astype(np.float32)
        x[u < 0.4] = -0.0
        return x
    if kind == "signed":
        return (u - 0.5).astype(np.float32)
    if kind == "close":  # the largest keys share their upper bits
        return (1.0 + np.floor(u * 64).astype(np.float32) * np.float32(2.0 ** -23)).astype(np.float32)
    return np.full(shape, 0.25, np.float32)


@pytest.mark.parametrize("kind", ["heavy", "ties", "zeros", "signed", "close", "equal"])
@pytest.mark.parametrize("unit", [1, 4])
@pytest.mark.parametrize("nkv", [1, 2, 8])
def test_lists(qsa, nkv, unit, kind):
    """Lengths of 0, 1, below a unit, at the budget and one past it, ragged tails, and long."""
    rng = qi.rng_for(50, salt=nkv * 10 + unit)
    keep, first, last = 64, 8, 16
    length = [0, 1, 3, 63, 64, 65, 67, 68, 71, 200, 1023, 1024, 4099, 5001]
    mass = draws(rng, kind, (len(length), nkv, 5004))
    sel, n_sel, st = call(qsa, mass, length, 5001, keep, first, last, unit)
    assert st == (0, 0)
    check(mass, length, keep, first, last, unit, sel, n_sel)


@pytest.mark.parametrize("keep,first,last", [(4, 0, 0), (4, 4, 0), (8, 4, 4), (400, 0, 400), (400, 400, 0), (1000, 12, 500),
                                             (4096, 0, 4)])
def test_budgets(qsa, keep, first, last):
    rng = qi.rng_for(51, salt=keep)
    length = [4098, 4100, 9999, 401]
    for unit in (1, 4):
        mass = draws(rng, "ties", (4, 2, 10000))
        sel, n_sel, st = call(qsa, mass, length, 9999, keep, first, last, unit)
        assert st == (0, 0)
        check(mass, length, keep, first, last, unit, sel, n_sel)


@pytest.mark.parametrize("kind", ["heavy", "zeros"])
@pytest.mark.parametrize("n,most,unit,keep", [(1, 300001, 1, 20000), (3, 262144, 4, 8192), (40, 40000, 4, 2048)])
def test_long_caches(qsa, n, most, unit, keep, kind):
    rng = qi.rng_for(52, salt=n)
    length = rng.integers(most // 2, most + 1, size=n)
    length[0] = most
    mass = draws(rng, kind, (n, 2, (most + 3) // 4 * 4))
    sel, n_sel, st = call(qsa, mass, length, most, keep, 16, 1024, unit)
    assert st == (0, 0)
    check(mass, length, keep, 16, 1024, unit, sel, n_sel)


def test_device_errors_leave_the_other_sequences(qsa):
    rng = qi.rng_for(53)
    mass = draws(rng, "heavy", (4, 2, 512))
    for bad in (np.nan, np.inf, -np.inf):
        m = mass.copy()
        m[1, 1, 77] = bad
        m[2, 0, 30] = bad          # a sequence that keeps everything: never read
        m[3, 0, 505] = bad         # past the length
        sel, n_sel, st = call(qsa, m, [500, 500, 64, 505], 512, 64, 4, 4, 4)
        assert st == (4, 1) and n_sel[1] == -7 and np.all(sel[1] == -5)
        for i, n in ((0, 500), (2, 64), (3, 505)):
            want = keep_units(np.nan_to_num(m[i]), n, 64, 4, 4, 4)
            assert n_sel[i] == len(want) and np.array_equal(sel[i, :len(want)], want)
    sel, n_sel, st = call(qsa, mass, [500, 513, 64, -1], 512, 64, 4, 4, 4)
    assert st[0] == 3 and st[1] in (1, 3) and n_sel[1] == -7 and n_sel[3] == -7
    check(mass[:1], [500], 64, 4, 4, 4, sel[:1], n_sel[:1])


def test_sums_that_overflow_are_nonfinite(qsa):
    mass = np.full((1, 2, 16), 3e38, np.float32)
    assert call(qsa, mass, [16], 16, 4, 0, 0, 1)[2] == (4, 0)


def test_graph(qsa):
    rng = qi.rng_for(54)
    mass = draws(rng, "ties", (3, 2, 2000))
    m, ln = dev(mass), dev(np.array([2000, 777, 100], np.int32))
    sel = torch.full((3, 203), -5, dtype=torch.int32, device="cuda")
    n_sel, st = torch.zeros(3, dtype=torch.int32, device="cuda"), qsa.new_status()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        qsa.qsa_evict_select(m, 2000, 2, ln, 3, 2000, 200, 4, 40, 4, sel, 203, n_sel, st)
    for length in ([2000, 777, 100], [1001, 203, 1999]):
        ln.copy_(dev(np.array(length, np.int32)))
        sel.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        check(mass, length, 200, 4, 40, 4, sel.cpu().numpy(), n_sel.cpu().numpy())
    assert qsa.qsa_read_status(st) == (0, 0)


def test_runs_that_shared_memory_does_not_hold(qsa):
    """A sequence whose share per CTA is past the cached keys: the mass is read again."""
    rng = qi.rng_for(55)
    most = 8 * 49152 + 2000
    mass = draws(rng, "heavy", (1, 1, (most + 3) // 4 * 4))
    mass[0, 0, ::3] = 0.0
    for length, unit, keep in ((most, 1, 30000), (most - 5, 1, 300000)):
        sel, n_sel, st = call(qsa, mass, [length], most, keep, 4, 64, unit)
        assert st == (0, 0)
        check(mass, [length], keep, 4, 64, unit, sel, n_sel)
    wide = draws(rng, "ties", (1, 1, 4 * most))
    sel, n_sel, st = call(qsa, wide, [4 * most], 4 * most, 8192, 4, 64, 4)
    assert st == (0, 0)
    check(wide, [4 * most], 8192, 4, 64, 4, sel, n_sel)
