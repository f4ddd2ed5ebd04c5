"""Edges of the step operators: pages and scales that no row sees, pools past 2^32 bytes, shared tables, odd groups,
heads that are not finite, and waits that give up."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev, f64
from step_cases import E4M3, Cache8, pool_8, ref_attend, scale_of, to_e4m3
from test_gpu_cache8 import SENT, call, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("rows,mask", [(1, "chain"), (20, "chain"), (300, "chain"), (9, "tree")])
@pytest.mark.parametrize("hd,page", [(128, 16), (256, 48)])
def test_pages_that_a_window_has_left_may_be_gone(qsa, hd, page, rows, mask):
    """Every page whose tokens are all past the first ones and before the window is taken out of the table, its scales
    and values are NaN: neither reaches a row, nor the status."""
    rng = qi.rng_for(100, salt=hd + rows)
    for n_first, window in ((0, 100), (4, 129), (17, 1), (200, 333)):
        c = Cache8(rng, [1500, 700], [rows, 2], 8, 2, hd, page, 16, mask, n_first=n_first, window=window)
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)
        for i in range(2):
            first_seen = int(c.ctx[i]) - (window - 1)
            for pg in range(c.table_len):
                if pg * page >= n_first and (pg + 1) * page <= first_seen:
                    at = int(c.table[i, pg]) * page
                    c.k[at:at + page], c.v[at:at + page] = 0x7F, 0xFF
                    c.ks[at // 16:(at + page) // 16] = np.nan
                    c.vs[at // 16:(at + page) // 16] = -1
                    c.table[i, pg] = -1 if pg % 2 else c.pages + 7
        again, lse2, st = call(qsa, c)
        assert st == (0, 0) and np.array_equal(again, out) and np.array_equal(lse2, lse)


@pytest.mark.parametrize("nq,nkv", [(65, 1), (3, 1), (9, 3), (17, 1), (33, 1), (96, 2)])
def test_odd_groups(qsa, nq, nkv):
    """Groups at the edges of the units' 8, 16, 32 and 64 rows, one row and a few a sequence."""
    for rows in ([1, 1, 1], [2, 7, 1]):
        rng = qi.rng_for(101, salt=nq)
        c = Cache8(rng, [400, 0, 129], rows, nq, nkv, 128, 16, 16, "tree")
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)


def test_one_table_for_several_sequences(qsa):
    """table_cols 0: sequences of different lengths read one cache."""
    rng = qi.rng_for(102)
    c = Cache8(rng, [900], [1], 16, 2, 256, 16, 16, "chain")
    n = 3
    lens = np.array([900, 333, 20], np.int32)
    q = qi.normal_bf16(rng, (n, 16 * 256), 1.5)
    d = c.device()
    out = torch.zeros((n, 4096), dtype=torch.int16, device="cuda")
    lse = torch.zeros((n, 16), device="cuda")
    st, ws = qsa.new_status(), qsa.new_cache8_workspace(n, n, 16, 2, 256)
    qsa.qsa_cache8_attn(dev(q), 4096, 16, 2, 256, d["k"], d["v"], d["ks"], d["vs"], 16, c.pages, 16, d["table"], c.table_len, 0,
                        dev(lens), dev(np.arange(n + 1, dtype=np.int32)), n, n, None, 0, 0, 0, 0.0625, out, 4096, lse, st, ws)
    assert qsa.qsa_read_status(st) == (0, 0)
    for i in range(n):
        c.ctx, c.q = lens[i:i + 1], q[i:i + 1]
        want, tol, wl, ltol = ref_attend(c, 0, 0.0625)
        got = f64(out.cpu().numpy().view(np.uint16)[i]).reshape(1, 16, 256)
        assert np.all(np.abs(got - want) <= tol) and np.all(np.abs(lse.cpu().numpy()[i] - wl[0]) <= ltol[0])


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_query_head_that_is_not_finite(qsa, bad):
    """It is NaN; the other heads and rows do not see it."""
    rng = qi.rng_for(103)
    for rows in ([1, 1], [20, 3]):
        c = Cache8(rng, [300, 200], rows, 8, 2, 128, 16, 16, "tree")
        out, lse, _ = call(qsa, c)
        c.q[0, 3 * 128 + 7] = qi.to_bf16_bits(np.array([bad], np.float32))[0]
        got, glse, st = call(qsa, c)
        assert st == (0, 0)
        here = np.zeros(got.shape, bool)
        here[0, 3 * 128:4 * 128] = True
        assert np.all(np.isnan(f64(got)[here])) and np.array_equal(got[~here], out[~here])
        assert np.isnan(glse[0, 3])


def test_pools_past_32_bits_of_bytes(qsa):
    """The last pages of pools of 4.6 GB: written and attended."""
    nq, nkv, hd, page, unit, n = 16, 8, 256, 16, 16, 2
    rng = qi.rng_for(104)
    pages = 140000
    width = nkv * hd
    k, v = (torch.zeros((pages * page, width), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages * page // unit, nkv), device="cuda") for _ in range(2))
    ctx, rows = np.array([100, 17], np.int32), np.array([30, 1], np.int32)
    table = (pages - 1 - np.arange(18, dtype=np.int32)).reshape(2, 9)
    start = np.array([0, 30, 31], np.int32)
    small_k, small_ks = pool_8(rng, 18 * page, nkv, hd, unit)
    small_v, small_vs = pool_8(rng, 18 * page, nkv, hd, unit)
    lo = (pages - 18) * page
    k[lo:].copy_(dev(small_k).view(-1, width))
    v[lo:].copy_(dev(small_v).view(-1, width))
    ks[lo // unit:].copy_(dev(small_ks))
    vs[lo // unit:].copy_(dev(small_vs))
    x = qi.normal_bf16(rng, (31, (nq + 2 * nkv) * hd), 2.0)
    c_t, s_t = qsa.qsa_rope_tables(200, 10000.0)
    xd = dev(x)
    q = torch.zeros((31, nq * hd), dtype=torch.int16, device="cuda")
    st = qsa.new_status()
    w = xd.shape[1]
    qsa.qsa_qkv_write(xd, w, nq, xd[:, nq * hd:], w, xd[:, (nq + nkv) * hd:], w, nkv, hd, None, None, 0.0, dev(c_t), dev(s_t), 200,
                      None, dev(ctx), dev(start), n, 31, k, v, ks, vs, unit, pages, page, dev(table), 9, 9, q, nq * hd, st)
    out = torch.zeros((31, nq * hd), dtype=torch.int16, device="cuda")
    lse = torch.zeros((31, nq), device="cuda")
    qsa.qsa_cache8_attn(q, nq * hd, nq, nkv, hd, k, v, ks, vs, unit, pages, page, dev(table), 9, 9, dev(ctx), dev(start), n, 31,
                        None, 0, 0, 0, 0.0625, out, nq * hd, lse, st, qsa.new_cache8_workspace(n, 31, nq, nkv, hd))
    assert qsa.qsa_read_status(st) == (0, 0)
    assert int(k[:lo].count_nonzero()) == 0 and int(ks[:lo // unit].count_nonzero()) == 0
    c = Cache8.__new__(Cache8)
    c.ctx, c.rows, c.nq, c.nkv, c.hd, c.page, c.unit, c.n, c.group = ctx, rows, nq, nkv, hd, page, unit, n, nq // nkv
    c.n_first = c.window = c.words = 0
    c.mask, c.row_start, c.n_rows = None, start, 31
    c.table = table - (pages - 18)
    c.k, c.v = (t[lo:].cpu().numpy().reshape(-1, nkv, hd) for t in (k, v))
    c.ks, c.vs = (t[lo // unit:].cpu().numpy() for t in (ks, vs))
    c.q = q.cpu().numpy().view(np.uint16)
    new = c.slots(0, np.arange(112, 128))  # a fresh block of V: its codes are exact
    true = f64(x[12:28, (nq + nkv) * hd:]).reshape(16, nkv, hd)
    s = scale_of(np.abs(true).max((0, 2)))
    assert np.array_equal(c.vs[new[0] // unit], s.astype(np.float32)) and np.array_equal(c.v[new], to_e4m3(true / s[None, :, None]))
    check(c, out.cpu().numpy().view(np.uint16), lse.cpu().numpy(), scale=0.0625)


@pytest.mark.parametrize("hd", [128, 256])
def test_attention_gives_up_and_recovers(qsa, hd):
    """A limit of a cycle makes a wait run out: the call returns, says so, and the next one is right."""
    default = qsa.qsa_wait_limit_cycles()
    for rows, nq in (([1, 1], 16), ([4, 1], 8), ([40, 9], 8), ([300, 2], 6)):
        c = Cache8(qi.rng_for(105, salt=hd), [5000, 40], rows, nq, 2, hd, 16, 16, "tree")
        want, lse, st = call(qsa, c)
        assert st == (0, 0)
        try:
            qsa.qsa_set_wait_limit_cycles(1)
            _, _, st = call(qsa, c)
        finally:
            qsa.qsa_set_wait_limit_cycles(default)
        assert st[0] == qsa.QSA_ERR_TIMEOUT and st[1] in (0, 1)
        got, lse2, st = call(qsa, c)
        assert st == (0, 0) and np.array_equal(got, want) and np.array_equal(lse2, lse)


def test_starts_that_do_not_ascend(qsa):
    """A start far above the others makes two sequences bad; the good ones, one split over many CTAs, keep their bits."""
    for hd, n in ((128, 4), (256, 40), (128, 700)):
        rng = qi.rng_for(106, salt=n)
        ctx, rows = np.full(n, 30), np.zeros(n, int)
        mid = n // 2
        ctx[-1], rows[-1] = 9001, 4
        c = Cache8(rng, ctx, rows, 8, 2, hd, 16, 16, "tree")
        want, wlse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, want, wlse)
        c.row_start[mid] = c.n_rows + 100
        out, lse, st = call(qsa, c)
        assert st[0] == 3 and st[1] in (mid - 1, mid)
        assert np.array_equal(out, want) and np.array_equal(lse, wlse)


def test_values_at_the_ends_of_the_type(qsa):
    """Codes of every kind: the largest, the smallest, both zeros, in K and in V."""
    rng = qi.rng_for(107)
    for hd in (128, 256):
        c = Cache8(rng, [600], [3], 8, 2, hd, 16, 16, "tree", q_std=0.02)
        codes = np.array([x for x in range(256) if x & 0x7F != 0x7F], np.uint8)
        c.k, c.v = rng.choice(codes, c.k.shape), rng.choice(codes, c.v.shape)
        assert not np.isnan(E4M3[c.v]).any()
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)
        assert SENT != 0
