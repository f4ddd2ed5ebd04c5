"""qsa_attn_mass against the plain form in 64 bits (cache_cases.ref_mass)."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev, ref_mass, ref_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def lse_of(c, scale):
    lse = np.zeros((c.n_rows, c.nq), np.float32)
    for i in range(c.n):
        r0 = int(c.row_start[i])
        lse[r0:r0 + int(c.rows[i])] = ref_tree(c, i, scale)[2].astype(np.float32)
    return lse


def call(qsa, c, lse, weight=None, carry=1.0, old=None, spare=8, q_pad=0, stream=None):
    scale = c.hd ** -0.5
    cols = (int((c.ctx + c.rows).max()) + 3) // 4 * 4 + spare
    if old is None:
        old = np.random.default_rng(5).random((c.n, c.nkv, cols), dtype=np.float32)
    mass = dev(old)
    st = qsa.new_status()
    row = c.nq * c.hd
    qb = np.zeros((c.n_rows, row + q_pad), np.uint16)
    qb[:, :row] = c.q
    w = None if weight is None else dev(weight)
    args = c.mass_args(dev(qb), row + q_pad)
    ld = dev(lse)
    torch.cuda.synchronize()
    qsa.qsa_attn_mass(*args, scale, ld, w, carry, mass, old.shape[2], st, stream=stream)
    torch.cuda.synchronize()
    return old, mass.cpu().numpy(), qsa.qsa_read_status(st)


def check(c, lse, weight, carry, old, got, seqs=None):
    for i in range(c.n) if seqs is None else seqs:
        kv = int(c.ctx[i] + c.rows[i])
        if c.rows[i] == 0:
            assert np.array_equal(got[i], old[i])
            continue
        r0 = int(c.row_start[i])
        want, tol = ref_mass(c, i, c.hd ** -0.5, lse[r0:r0 + int(c.rows[i])], weight, carry, old[i])
        err = np.abs(got[i][:, :kv] - want)
        assert np.all(err <= tol), f"sequence {i}: {np.max(err / tol)} of the bound"
        assert np.array_equal(got[i][:, kv:], old[i][:, kv:]), "entries past the tokens were written"


@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
@pytest.mark.parametrize("nq,nkv,hd,page", [(16, 2, 256, 16), (8, 1, 128, 7), (6, 2, 128, 64), (24, 2, 256, 1),
                                            (32, 8, 128, 16)])
def test_ragged_batch(qsa, nq, nkv, hd, page, mask):
    rng = qi.rng_for(40, salt=nq * 100 + hd + page)
    c = Cache(rng, [0, 1, 127, 128, 129, 300, 90, 255], [3, 1, 1, 5, 0, 40, 38, 2], nq, nkv, hd, page, mask, gaps=1)
    lse = lse_of(c, hd ** -0.5)
    old, got, st = call(qsa, c, lse, q_pad=8)
    assert st == (0, 0)
    check(c, lse, None, 1.0, old, got)


@pytest.mark.parametrize("carry", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("hd", [128, 256])
def test_weights_and_carry(qsa, hd, carry):
    """Row weights (zero ones on rows of NaN), carry 0 over NaN mass, drafted
    tokens' old entries NaN: none of it shows."""
    rng = qi.rng_for(41, salt=hd)
    c = Cache(rng, [200, 33], [9, 20], 8, 2, hd, 16, "tree")
    lse = lse_of(c, hd ** -0.5)
    weight = rng.choice([0.0, 1.0, 0.5], size=c.n_rows).astype(np.float32)
    weight[3], weight[12] = 0.0, 0.0
    c.q[3] = 0x7FC0
    lse[12] = np.nan
    old = rng.random((2, 2, 256), dtype=np.float32)
    for i in range(2):
        old[i, :, c.ctx[i]:c.ctx[i] + c.rows[i]] = np.nan
    if carry == 0.0:
        old[0, :, :200] = np.nan
    old, got, st = call(qsa, c, lse, weight, carry, old)
    assert st == (0, 0)
    q3 = c.q[3].copy()
    c.q[3] = 0
    check(c, lse, weight, carry, np.nan_to_num(old), np.nan_to_num(got))
    c.q[3] = q3
    for i in range(2):
        assert np.all(np.isfinite(got[i][:, :c.ctx[i] + c.rows[i]]))


@pytest.mark.parametrize("rows,mask", [(70, "tree"), (129, "tree"), (300, "chain")])
@pytest.mark.parametrize("hd", [128, 256])
def test_many_rows(qsa, hd, rows, mask):
    rng = qi.rng_for(42, salt=rows + hd)
    c = Cache(rng, [140, 0], [rows, 9], 6, 2, hd, 16, mask)
    lse = lse_of(c, hd ** -0.5)
    old, got, st = call(qsa, c, lse, carry=0.5)
    assert st == (0, 0)
    check(c, lse, None, 0.5, old, got)


def test_long_context_and_rows_that_see_nothing(qsa):
    rng = qi.rng_for(43)
    c = Cache(rng, [9000, 0, 40], [2, 3, 1], 16, 2, 256, 16, "tree")
    c.set_bits(1, np.array([[0, 0, 0], [1, 0, 0], [0, 0, 0]], bool))
    lse = lse_of(c, 256 ** -0.5)
    assert np.all(np.isneginf(lse[2])) and np.all(np.isneginf(lse[4]))
    old, got, st = call(qsa, c, lse)
    assert st == (0, 0)
    check(c, lse, None, 1.0, old, got)


def test_total_is_one_per_row_and_head(qsa):
    """With the attention's own lse, a sequence's mass of one step adds up to its
    rows times its group's heads."""
    rng = qi.rng_for(44)
    c = Cache(rng, [1000, 17], [5, 3], 16, 2, 256, 16, "tree")
    out = torch.zeros((c.n_rows, c.nq * c.hd), dtype=torch.int16, device="cuda")
    lse = torch.zeros((c.n_rows, c.nq), dtype=torch.float32, device="cuda")
    st = qsa.new_status()
    qsa.qsa_tree_attn(*c.tree_args(dev(c.q), c.nq * c.hd), c.hd ** -0.5, out, c.nq * c.hd, lse, st,
                      qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd))
    old = np.zeros((2, 2, 1008), np.float32)
    _, got, s2 = call(qsa, c, lse.cpu().numpy(), old=old)
    assert qsa.qsa_read_status(st) == (0, 0) and s2 == (0, 0)
    # each p is off by under 1e-4 (2 delta + lse's own error at these sizes)
    assert np.allclose(got.sum(2, dtype=np.float64), np.array([[5 * 8] * 2, [3 * 8] * 2]), rtol=1e-4)


def test_device_errors_leave_the_other_sequences(qsa):
    rng = qi.rng_for(45)
    for kind in ("context", "cols", "mask", "page"):
        c = Cache(rng, [50, 60, 70], [4, 40, 4], 8, 2, 128, 16, "tree")
        lse = lse_of(c, 128 ** -0.5)
        old, good, st = call(qsa, c, lse)
        assert st == (0, 0)
        if kind == "context":
            c.ctx[1] = c.table_len * 16 - 39
        elif kind == "cols":
            old = np.ascontiguousarray(old[:, :, :96])
        elif kind == "mask":
            c.mask, c.words = np.ascontiguousarray(c.mask[:, :1]), 1
        else:
            c.table[1, 2] = -3
        _, got, st = call(qsa, c, lse, old=old)
        assert st == ((6, 1) if kind == "page" else (3, 1))
        for i in (0, 2):
            assert np.array_equal(got[i], good[i][:, :old.shape[2]])
        if kind != "page":
            assert np.array_equal(got[1], old[1])


def test_repeats_and_graphs(qsa):
    rng = qi.rng_for(46)
    c = Cache(rng, [3000, 9], [7, 20], 16, 2, 256, 16, "tree")
    lse = lse_of(c, 256 ** -0.5)
    old, got, _ = call(qsa, c, lse)
    again, stream = call(qsa, c, lse)[1], call(qsa, c, lse, stream=torch.cuda.Stream())[1]
    assert np.array_equal(got, again) and np.array_equal(got, stream)
    mass, st, ld = dev(old), qsa.new_status(), dev(lse)
    args = c.mass_args(dev(c.q), c.nq * c.hd)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        qsa.qsa_attn_mass(*args, c.hd ** -0.5, ld, None, 1.0, mass, old.shape[2], st)
    mass.copy_(dev(old))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(mass.cpu().numpy(), got) and qsa.qsa_read_status(st) == (0, 0)
