"""The cache operators at the calls between the ordinary ones: more sequences than a
CTA has threads, groups of heads wider than a tile of rows, sequences of very unequal
width in one call, scales of either sign, shared workspaces, several host threads.
Plain forms and tolerances are those of cache_cases."""
import threading

import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev, f64, keep_units, ref_mass, ref_tree
from test_gpu_compact import Pool
from test_gpu_compact import call as compact_call
from test_gpu_compact import same, whole_blocks
from test_gpu_compact import want as compact_want
from test_gpu_evict import call as evict_call
from test_gpu_mass import call as mass_call
from test_gpu_mass import check as mass_check
from test_gpu_mass import lse_of
from test_gpu_tree import call as tree_call
from test_gpu_tree import check as tree_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def both(qsa, c):
    out, lse, st = tree_call(qsa, c)
    assert st == (0, 0)
    tree_check(c, out, lse)
    given = lse_of(c, c.hd ** -0.5)
    old, got, st = mass_call(qsa, c, given, carry=0.5)
    assert st == (0, 0)
    mass_check(c, given, None, 0.5, old, got)


@pytest.mark.parametrize("n,hd", [(1, 128), (449, 256), (1000, 128)])
def test_many_sequences(qsa, n, hd):
    """Sequences of 0 to 40 tokens, some without rows."""
    rng = qi.rng_for(60, salt=n)
    c = Cache(rng, rng.integers(0, 40, n), rng.integers(0, 4, n), 2, 1, hd, 8, "tree")
    both(qsa, c)


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("nq,nkv,rows", [(130, 1, [1, 3]), (262, 2, [2, 1]), (300, 1, [1, 2]), (63, 21, [5, 40]), (5, 1, [33, 52])])
def test_wide_and_odd_groups(qsa, nq, nkv, rows, hd):
    """Groups of 130 and 300 heads end inside a turn of pairs and inside a tile of rows."""
    c = Cache(qi.rng_for(61, salt=nq + hd), [200, 9], rows, nq, nkv, hd, 16, "tree")
    both(qsa, c)


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("mask", ["tree", "chain"])
@pytest.mark.parametrize("rows", [[300, 1, 0, 20], [57, 56, 1], [49, 0, 1]])
def test_unequal_widths(qsa, rows, mask, hd):
    """Means of 4, 2 and 1 tiles of rows a sequence, whose own counts are 19, 1 and 0."""
    c = Cache(qi.rng_for(62, salt=len(rows) + hd), [700, 90, 5, 1][:len(rows)], rows, 16, 2, hd, 16, mask)
    both(qsa, c)


@pytest.mark.parametrize("hd", [128, 256])
def test_units_shorter_than_a_share(qsa, hd):
    """Far more units than CTAs, each of one to six tiles."""
    rng = qi.rng_for(63, salt=hd)
    c = Cache(rng, rng.integers(0, 400, 60), rng.integers(1, 4, 60), 8, 8, hd, 16, "tree")
    both(qsa, c)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 0.3])
@pytest.mark.parametrize("hd", [128, 256])
def test_scales(qsa, hd, scale):
    c = Cache(qi.rng_for(64, salt=hd), [150, 20], [5, 19], 8, 2, hd, 16, "tree", q_std=0.5)
    out, lse, st = tree_call(qsa, c, scale=scale)
    assert st == (0, 0)
    tree_check(c, out, lse, scale=scale)
    given = np.zeros((c.n_rows, c.nq), np.float32)
    for i in range(c.n):
        r0 = int(c.row_start[i])
        given[r0:r0 + int(c.rows[i])] = ref_tree(c, i, scale)[2].astype(np.float32)
    row, cols = c.nq * c.hd, 176
    old = np.random.default_rng(6).random((c.n, c.nkv, cols), dtype=np.float32)
    mass, st = dev(old), qsa.new_status()
    qsa.qsa_attn_mass(*c.mass_args(dev(c.q), row), scale, dev(given), None, 1.0, mass, cols, st)
    assert qsa.qsa_read_status(st) == (0, 0)
    got = mass.cpu().numpy()
    for i in range(c.n):
        r0, m, kv = int(c.row_start[i]), int(c.rows[i]), int(c.ctx[i] + c.rows[i])
        want, tol = ref_mass(c, i, scale, given[r0:r0 + m], None, 1.0, old[i])
        assert np.all(np.abs(got[i][:, :kv] - want) <= tol)


def test_calls_without_rows(qsa):
    """No sequence has rows: nothing is written."""
    c = Cache(qi.rng_for(65), [100, 7], [0, 0], 8, 2, 128, 16, "chain", gaps=3)
    out, lse, st = tree_call(qsa, c)
    assert st == (0, 0) and np.all(out == 0x7FAB) and np.all(lse == 123.0)
    old, got, st = mass_call(qsa, c, np.zeros((c.n_rows, c.nq), np.float32))
    assert st == (0, 0) and np.array_equal(old, got)


def test_nonfinite_values_of_wide_trees(qsa):
    """Values that are not finite among drafted tokens, seen by some tiles of rows and not by others."""
    for hd in (128, 256):
        rng = qi.rng_for(66, salt=hd)
        c = Cache(rng, [130, 40], [80, 3], 16, 2, hd, 16, "tree")
        at = c.slots(0, 130 + np.array([5, 50, 79]))
        c.v[at[0], 3], c.v[at[1], hd + 7], c.v[at[2], hd - 1] = 0x7F80, 0x7FC0, 0xFF80
        out, lse, st = tree_call(qsa, c)
        assert st == (0, 0)
        tree_check(c, out, lse)


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80])
def test_keys_that_are_not_finite(qsa, hd, bad):
    """Every key of the first tiles, one in the middle, or a drafted one: each row that
    sees one gets NaN (its logit may be an infinity of either sign, or NaN), and lse too."""
    rng = qi.rng_for(70, salt=hd)
    for where in ("first", "one", "drafted"):
        c = Cache(rng, [400, 60], [9, 3], 8, 2, hd, 16, "tree")
        if where == "first":
            c.k[c.slots(0, np.arange(200))] = bad
        elif where == "one":
            c.k[c.slots(0, np.array([250])), 5] = bad
        else:
            c.k[c.slots(0, np.array([403])), hd + 1] = bad
        out, lse, st = tree_call(qsa, c)
        assert st == (0, 0)
        tree_check(c, out, lse)


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("at", [0, 31, 32, 33, 63, 64, 95, 96, 127, 191, 192, 250])
def test_a_token_far_above_the_others(qsa, hd, at):
    """One key some 200 log2 units above the rest, at the edges of columns and tiles, and a
    second one 30 below it further on."""
    rng = qi.rng_for(72, salt=hd + at)
    c = Cache(rng, [260], [3], 8, 2, hd, 16, "tree", q_std=0.25)
    scale = hd ** -0.5
    for g in range(2):
        q = f64(c.q[0]).reshape(8, hd)[4 * g:4 * g + 4].sum(0)
        for t, units in ((at, 200.0), (min(at + 70, 259), 170.0)):
            k = q / (q @ q) * 4 * units * np.log(2) / scale
            c.k[c.slots(0, np.array([t]))[0], g * hd:(g + 1) * hd] = qi.to_bf16_bits(k.astype(np.float32))
    out, lse, st = tree_call(qsa, c)
    assert st == (0, 0)
    tree_check(c, out, lse)


def test_refuses_tensors_of_another_device(qsa, monkeypatch):
    c = Cache(qi.rng_for(71), [40], [2], 8, 2, 128, 16, "tree")
    args = c.tree_args(dev(c.q), c.nq * c.hd)
    out, st = torch.zeros((2, 1024), dtype=torch.int16, device="cuda"), qsa.new_status()
    ws = qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd)
    x = torch.zeros(64, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0"):
        qsa.qsa_tree_attn(*args, 1.0, out, 1024, None, st, ws)
    with pytest.raises(ValueError, match="cuda:0"):
        qsa.qsa_attn_mass(*c.mass_args(args[0], 1024), 1.0, x, None, 1.0, x, 64, st)
    with pytest.raises(ValueError, match="cuda:0"):
        qsa.qsa_evict_select(x, 64, 1, x, 1, 64, 4, 0, 0, 4, x, 64, x, st)
    with pytest.raises(ValueError, match="cuda:0"):
        qsa.qsa_cache_compact(x, x, 8, 1, x, 1, 1, 1, x, 1, x, 1, 1, None, None, 0, 0, None, None, st)


def test_two_graphs_share_a_workspace(qsa):
    """Two captured calls of different shapes use the same workspace, replayed in turn on one stream."""
    cs = [Cache(qi.rng_for(67, salt=i), [3000 - 900 * i, 50], [6, 20 * i + 1], 16, 2, 256, 16, "tree") for i in range(2)]
    want = [tree_call(qsa, c)[:2] for c in cs]
    ws = max((qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd) for c in cs), key=lambda w: w.numel())
    graphs, keep = [], []
    for c in cs:
        row = c.nq * c.hd
        out = torch.zeros((c.n_rows, row), dtype=torch.int16, device="cuda")
        lse = torch.zeros((c.n_rows, c.nq), dtype=torch.float32, device="cuda")
        st, args = qsa.new_status(), c.tree_args(dev(c.q), row)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            qsa.qsa_tree_attn(*args, c.hd ** -0.5, out, row, lse, st, ws)
        graphs.append(g)
        keep.append((out, lse, st, args))
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (out, lse, st, _), (o, l) in zip(keep, want):
        assert qsa.qsa_read_status(st) == (0, 0)
        assert np.array_equal(out.cpu().numpy().view(np.uint16), o) and np.array_equal(lse.cpu().numpy(), l)


def test_mass_accumulates_in_a_graph(qsa):
    """Three replays add three times the weights of one (carry 1), in the bits of three calls."""
    c = Cache(qi.rng_for(68), [500, 30], [40, 2], 16, 2, 256, 16, "tree")
    given = lse_of(c, c.hd ** -0.5)
    old, once, st = mass_call(qsa, c, given)
    cur = once
    for _ in range(2):
        _, cur, _ = mass_call(qsa, c, given, old=cur)
    mass, ld, stat = dev(old), dev(given), qsa.new_status()
    args = c.mass_args(dev(c.q), c.nq * c.hd)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        qsa.qsa_attn_mass(*args, c.hd ** -0.5, ld, None, 1.0, mass, old.shape[2], stat)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert qsa.qsa_read_status(stat) == (0, 0)
    got = mass.cpu().numpy()
    for i in range(c.n):  # a drafted token's mass starts at zero in every call
        assert np.array_equal(got[i], cur[i])


def test_host_threads_on_their_own_streams(qsa):
    """Mass, eviction and compaction from four threads at once, ten calls each."""
    c = Cache(qi.rng_for(69), [900, 40], [5, 70], 16, 2, 256, 16, "tree")
    given = lse_of(c, c.hd ** -0.5)
    rng = np.random.default_rng(7)
    mass = (rng.random((3, 2, 20000), dtype=np.float32) ** 9).astype(np.float32)
    length = np.array([20000, 4097, 300], np.int32)
    pool = Pool(qi.rng_for(69, salt=1), 3, 600, 16, 256, 2, True)
    lists = [np.arange(0), np.array([77]), np.arange(8, 552)]
    first_mass = mass_call(qsa, c, given)
    first_list = evict_call(qsa, mass, length, 20000, 2048, 16, 128, 4)
    moved = compact_want(pool, lists, None)
    errors, gate = [], threading.Barrier(4)

    def worker(i):
        try:
            torch.cuda.set_device(0)
            s = torch.cuda.Stream()
            gate.wait()
            for _ in range(10):
                if i % 3 == 0:
                    assert np.array_equal(mass_call(qsa, c, given, stream=s)[1], first_mass[1])
                elif i % 3 == 1:
                    got = evict_call(qsa, mass, length, 20000, 2048, 16, 128, 4, stream=s)
                    assert np.array_equal(got[0], first_list[0]) and np.array_equal(got[1], first_list[1])
                else:
                    got = compact_call(qsa, pool, lists, None, stream=s)
                    assert got[4] == (0, 0)
                    same(got[:4], moved)
        except Exception as e:
            errors.append(repr(e))

    ts = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


def test_lists_for_many_sequences(qsa):
    """A thousand short caches, and lists of caches of every length around the budget."""
    rng = np.random.default_rng(8)
    length = np.concatenate([np.arange(0, 80), rng.integers(0, 300, 920)]).astype(np.int32)
    mass = rng.random((1000, 2, 300), dtype=np.float32)
    for unit, keep, first, last in ((1, 37, 3, 5), (4, 40, 4, 8)):
        sel, n_sel, st = evict_call(qsa, mass, length, 300, keep, first, last, unit)
        assert st == (0, 0)
        for i in range(1000):
            want = keep_units(mass[i], int(length[i]), keep, first, last, unit)
            assert n_sel[i] == len(want) and np.array_equal(sel[i, :len(want)], want)


@pytest.mark.parametrize("n,tokens,page,width,nkv", [(40, 300, 16, 512, 2), (160, 90, 7, 136, 1), (12, 900, 64, 1024, 8)])
def test_moves_of_many_sequences(qsa, n, tokens, page, width, nkv):
    """More slices than SMs, with block keys; lists of every length from nothing on."""
    rng = qi.rng_for(73, salt=n)
    p = Pool(rng, n, tokens, page, width, nkv, True)
    lists = [whole_blocks(rng, tokens, int(rng.integers(0, tokens // 4 + 1)) if i else 0, 0) for i in range(n)]
    got = compact_call(qsa, p, lists, None)
    assert got[4] == (0, 0)
    same(got[:4], compact_want(p, lists, None))
