"""Weights of qsa_cache8_attn beside one that dominates, as a first token's often does, with a V that is small: the many
small ones are the output.

The tolerance is that of drafted-row attention over a bf16 cache (cache_cases.ref_tree) on the values that the cache
stands for, beside which the logits' bound (step_cases) counts what q's two terms lose: 2^-8 of every weight, nothing of
the largest one.  A weight's terms are off by 2^-9 of it and 2^-11 for its f16, or by 2^-19 where the row's largest is
2^8, or up to 2^14: as much more as it is more than 2^10 above the others of its tile.  One that has 0.99 of the sum of
65536 is 2^22.6 above the others' mean and 2^18 above theirs (of 32 normal logits the largest is some 2^3 above the mean,
the least of four such less), so at 2^14: 2^16 * 2^-33 of it together, within the (2^-8 - 2^-9 - 2^-11) * 0.01 that is
left.  One of 0.9 among 16384 is 2^17.9 above the mean, so at 2^12 or more: 2^14 * 2^-31 beside 0.1.
"""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import BF, U, dev, f64
from step_cases import Cache8, ref_attend, to_e4m3
from test_gpu_cache8 import call, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def dominated(rng, tokens, rows, group, hd, weight, large):
    """A sequence whose token `large` has about `weight` of every row's sum, logits N(0, 1) else, V N(0, 1) + 0.3 and of the
    token `large` 0.05 N(0, 1)."""
    c = Cache8(rng, [tokens - rows], [rows], group, 1, hd, 64, 64, "chain", q_std=1.5)
    q = f64(c.q).reshape(rows * group, hd)
    k = rng.standard_normal((tokens, hd)) / 1.5
    top = np.log(weight / (1 - weight) * tokens) + 0.5
    k[large] = np.linalg.pinv(q) @ np.full(rows * group, top * hd ** 0.5)
    v = rng.standard_normal((tokens, hd)) + 0.3
    v[large] = 0.05 * rng.standard_normal(hd)
    at = c.slots(0, np.arange(tokens))
    for pool, scales, x in ((c.k, c.ks, k), (c.v, c.vs, v)):
        blocks = -(-tokens // 64)
        pad = np.zeros((blocks * 64, hd))
        pad[:tokens] = x
        s = np.exp2(np.ceil(np.log2(np.abs(pad).reshape(blocks, -1).max(1) / 448)))
        scales[at[::64] // 64, 0] = s
        pool[at, 0] = to_e4m3(pad / np.repeat(s, 64)[:, None])[:tokens]
    return c


def bound_of_bf16(c, scale):
    """ref_attend's outputs with the bound of bf16 weights."""
    want, _, lse, ltol = ref_attend(c, 0, scale)
    m = int(c.rows[0])
    q = f64(c.q).reshape(m, c.nq, c.hd)
    k, v, _, _ = c.kv(0)
    k, v, vis = k[:, 0], v[:, 0], c.sees(0)
    tol = np.zeros(want.shape)
    for j in range(m):
        kj, vj, n = k[vis[j]], v[vis[j]], int(vis[j].sum())
        s = (q[j] @ kj.T) * scale
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        delta = scale * np.max((c.hd + 8) * 2 * U * (np.abs(q[j]) @ np.abs(kj).T)
                               + 2.0 ** -17 * np.abs(q[j]).max(1, keepdims=True) * np.abs(kj).sum(1)[None], axis=1)
        tol[j] = (BF + 4 * delta[:, None] + 2.0 ** -20 + 2 * n * U) * (p @ np.abs(vj)) + BF * np.abs(want[j])
    return want, tol, lse, ltol


# The sequence many times over, so that units lie whole in CTAs and across them; units of 8, 16, 32 and 64 rows.
@pytest.mark.parametrize("rows,group", [(1, 8), (2, 8), (4, 8), (8, 8)])
@pytest.mark.parametrize("tokens,weight", [(16384, 0.5), (16384, 0.9), (16384, 0.99), (65536, 0.5), (65536, 0.9), (65536, 0.99)])
def test_small_weights_beside_a_large_one(qsa, tokens, weight, rows, group):
    for hd, large in ((128, 0), (256, 0), (128, tokens // 2 + 77), (256, tokens - 200)):
        rng = qi.rng_for(112, salt=tokens + hd + rows + int(weight * 100))
        c = dominated(rng, tokens, rows, group, hd, weight, large)
        scale = hd ** -0.5
        want, tol, wl, ltol = bound_of_bf16(c, scale)
        n, d = 170, c.device()
        q = dev(np.tile(c.q, (n, 1)))
        out = torch.zeros((n * rows, group * hd), dtype=torch.int16, device="cuda")
        lse = torch.zeros((n * rows, group), device="cuda")
        st, ws = qsa.new_status(), qsa.new_cache8_workspace(n, n * rows, group, 1, hd)
        ctx, start = dev(np.full(n, tokens - rows, np.int32)), dev(np.arange(n + 1, dtype=np.int32) * rows)
        qsa.qsa_cache8_attn(q, group * hd, group, 1, hd, d["k"], d["v"], d["ks"], d["vs"], 64, c.pages, 64, d["table"],
                            c.table_len, 0, ctx, start, n, n * rows, None, 0, 0, 0, scale, out, group * hd, lse, st, ws)
        assert qsa.qsa_read_status(st) == (0, 0)
        got = f64(out.cpu().numpy().view(np.uint16)).reshape(n, rows, group, hd)
        err = np.abs(got - want[None]) / tol[None]
        assert err.max() <= 1, (hd, large, err.max())
        assert np.all(np.abs(lse.cpu().numpy().reshape(n, rows, group) - wl[None]) <= ltol[None])


@pytest.mark.parametrize("log2", [-80, -60, 38, 100])
def test_v_scales_at_the_ends_of_their_range(qsa, log2):
    """V's scales far below and above 1, all alike: the bound is of the outputs' own size."""
    rng = qi.rng_for(119, salt=log2 + 200)
    for hd, rows in ((128, 1), (256, 12)):
        c = Cache8(rng, [900, 40], [rows, 1], 8, 2, hd, 16, 16, "tree")
        c.vs = np.ldexp(c.vs, log2).astype(np.float32)
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)
