"""What a bad sequence, or a wait that runs out, leaves of the others and of the status word."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev
from test_gpu_mass import call as mass_call
from test_gpu_tree import call as tree_call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("n", [3, 40, 500])
def test_starts_that_do_not_ascend_leave_the_good_sequences(qsa, n, hd):
    """A start far above the others, in the middle, makes two sequences bad; one behind them
    owns rows 0..3 of a context that many CTAs share, and another the rows after those."""
    rng = qi.rng_for(80, salt=n + hd)
    ctx, rows = np.full(n, 30), np.zeros(n, int)
    mid = n // 2
    good = [n - 1] if n == 3 else [mid + 1, n - 1]
    for k, i in enumerate(good):
        ctx[i], rows[i] = (9001, 4) if k == 0 else (20, 2)
    c = Cache(rng, ctx, rows, 8, 2, hd, 16, "tree")
    want, wlse, st = tree_call(qsa, c)
    assert st == (0, 0)
    lse = np.where(np.isfinite(wlse), wlse, 0).astype(np.float32)
    old, wmass, st = mass_call(qsa, c, lse)
    assert st == (0, 0)
    c.row_start[mid] = 10 * n + 100  # past n_rows: the sequences on either side contradict themselves
    out, glse, st = tree_call(qsa, c)
    assert st[0] == 3 and st[1] in (mid - 1, mid)
    assert np.array_equal(out, want) and np.array_equal(glse, wlse)
    _, mass, st = mass_call(qsa, c, lse, old=old)
    assert st[0] == 3 and st[1] in (mid - 1, mid)
    assert np.array_equal(mass, wmass)


def test_many_rows_of_a_bad_sequence(qsa):
    """Twenty thousand sequences, one of which claims thirty thousand rows that it may not
    have, beside starts that do not ascend: rows that no sequence has cost the join little."""
    n, more = 20000, 30000
    c = Cache(qi.rng_for(88), np.full(n, 3), np.zeros(n, int), 8, 2, 128, 16, "chain")
    ctx, rows = c.ctx, c.rows
    ctx[n - 2], rows[n - 2], rows[n - 1] = 9001, 4, 1
    c = Cache(qi.rng_for(89), ctx, rows, 8, 2, 128, 16, "chain")
    c.q = np.concatenate([c.q, np.zeros((more, 8 * 128), np.uint16)])
    c.n_rows += more
    want, wlse, st = tree_call(qsa, c)
    assert st == (0, 0)
    c.row_start[n // 2] = c.n_rows - 1  # the one before has all rows, and a context too long for its table
    c.ctx[n // 2 - 1] = c.table_len * 16
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    out, lse, st = tree_call(qsa, c)
    t1.record()
    t1.synchronize()
    assert st[0] == 3 and st[1] in (n // 2 - 1, n // 2)
    assert np.array_equal(out, want) and np.array_equal(lse, wlse)
    assert t0.elapsed_time(t1) < 5000  # with the copies


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("rows", [1, 60])
def test_a_timeout_names_a_sequence_of_the_call(qsa, hd, rows):
    """Most CTAs have no share of two short sequences: they have nothing to wait for, and
    those that do name a sequence with rows."""
    default = qsa.qsa_wait_limit_cycles()
    c = Cache(qi.rng_for(81, salt=hd + rows), [7, 300, 9, 40], [0, rows, 0, 2], 8, 2, hd, 16, "tree")
    lse = dev(np.zeros((c.n_rows, c.nq), np.float32))
    args = c.mass_args(dev(c.q), c.nq * hd)
    targs = c.tree_args(dev(c.q), c.nq * hd)
    out = torch.zeros((c.n_rows, c.nq * hd), dtype=torch.int16, device="cuda")
    ws = qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, hd)
    mass = torch.zeros((c.n, c.nkv, 400), dtype=torch.float32, device="cuda")
    try:
        qsa.qsa_set_wait_limit_cycles(1)
        for _ in range(10):
            st = qsa.new_status()
            qsa.qsa_attn_mass(*args, hd ** -0.5, lse, None, 1.0, mass, 400, st)
            st = qsa.qsa_read_status(st)
            assert st[0] == 5 and st[1] in (1, 3)
            st = qsa.new_status()
            qsa.qsa_tree_attn(*targs, hd ** -0.5, out, c.nq * hd, None, st, ws)
            st = qsa.qsa_read_status(st)
            assert st[0] == 5 and st[1] in (1, 3)
    finally:
        qsa.qsa_set_wait_limit_cycles(default)


def test_calls_with_nothing_to_do_take_no_tensors(qsa):
    """As in the library's other calls: no sequences or rows and no tensors is no error, and
    the same call with rows is refused."""
    def calls(n):
        yield lambda: qsa.qsa_tree_attn(None, 0, 8, 2, 128, None, None, 0, 16, None, 0, 0, None, None, n, n, None, 0, 1.0, None,
                                        0, None, None, None)
        yield lambda: qsa.qsa_attn_mass(None, 0, 8, 2, 128, None, 0, 16, None, 0, 0, None, None, n, n, None, 0, 1.0, None, None,
                                        1.0, None, 0, None)
        yield lambda: qsa.qsa_evict_select(None, 0, 2, None, n, 0, 4, 0, 0, 4, None, 0, None, None)
        yield lambda: qsa.qsa_cache_compact(None, None, 512, 0, None, 0, 0, 16, None, 0, None, n, n, None, None, 0, 0, None,
                                            None, None)
    for f in calls(0):
        f()
    for f in calls(1):
        with pytest.raises(qsa.QsaError):
            f()
