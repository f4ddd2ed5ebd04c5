"""What goes on over a cache that was cut back: the indexer's steps (pool the next block,
score, select, in their own calls and in the one-launch ones), the token list, the gather
and the sparse attention, against the oracle over the surviving tokens."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import BF, U, dev, f64, keep_units
from qsa_cases import EPS, THETA, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("length", [902, 1203, 2304])
def test_steps_over_a_cut_cache(qsa, orc, length):
    """Eight tokens, one at a time, behind a cache cut from `length` to 512 and its tail: two
    blocks are completed on the way, at cached indices that are not their positions."""
    rng = qi.rng_for(90, salt=length)
    nq, nkv, hd, page, budget, select = 8, 2, 128, 16, 512, 128
    width, row, scale, steps = nkv * hd, nq * hd, hd ** -0.5, 8
    most = (length + steps + page - 1) // page * page
    pages = most // page
    table = rng.permutation(pages).astype(np.int32)[None]
    k, v = qi.normal_bf16(rng, (most, width)), qi.normal_bf16(rng, (most, width))
    raw = qi.raw_keys(rng, length + steps)
    fq = qi.fused_qk(rng, steps)
    qw, kw = qi.norm_weights(rng)
    cos_t, sin_t = qsa.qsa_rope_tables(most, THETA)
    cd, sd, qwd, kwd, td = dev(cos_t), dev(sin_t), dev(qw), dev(kw), dev(table)

    def slots(t):
        t = np.asarray(t)
        return table[0, t // page].astype(np.int64) * page + t % page

    kp, vp = np.zeros_like(k), np.zeros_like(v)
    kp[slots(np.arange(length))], vp[slots(np.arange(length))] = k[:length], v[:length]
    kd, vd, rawd = dev(kp), dev(vp), dev(raw)
    blocks, cols = most // 4, (most // 4 + 3) // 4 * 4
    keys = torch.zeros((blocks, 128), dtype=torch.int16, device="cuda")
    qsa.qsa_pool_blocks(rawd, 128, 0, length // 4, kwd, cd, sd, most, EPS, keys)
    true_keys = orc.pool_blocks(raw, 128, 0, (length + steps) // 4, kw, cos_t, sin_t, EPS)
    mass = rng.random((1, nkv, most), dtype=np.float32)
    sel = torch.full((1, budget + 3), -1, dtype=torch.int32, device="cuda")
    n_sel, st = torch.zeros(1, dtype=torch.int32, device="cuda"), qsa.new_status()
    qsa.qsa_evict_select(dev(mass), most, nkv, dev(np.array([length], np.int32)), 1, most, budget, 4, 64, 4, sel, budget + 3,
                         n_sel, st)
    kept = keep_units(mass[0], length, budget, 4, 64, 4)
    assert np.array_equal(sel.cpu().numpy()[0, :int(n_sel.item())], kept)
    qsa.qsa_cache_compact(kd, vd, width, pages, td, pages, pages, page, sel, budget + 3, n_sel, 1, budget + 3, None, None, 0,
                          nkv, keys, None, st)
    assert qsa.qsa_read_status(st) == (0, 0)
    gone = length - len(kept)  # tokens dropped
    assert gone > 0 and gone % 4 == 0
    tokens = list(kept)        # the cache's tokens, by their places in the sequence
    ws = qsa.new_decode_workspace(1, most)
    stepped = torch.zeros_like(keys)
    for i in range(steps):
        true, at = length + i, length + i - gone
        tokens.append(true)
        assert len(tokens) == at + 1
        kd[slots(at)], vd[slots(at)] = dev(k[true:true + 1])[0], dev(v[true:true + 1])[0]
        ends, block = (at + 1) % 4 == 0, at // 4
        seen = (at + 1) // 4
        want_keys = true_keys[np.asarray(tokens[:4 * seen:4], int) // 4]
        # each path pools, scores and selects on its own copy of the keys
        q = dev(fq[i:i + 1])
        block_raw = rawd[true - 3:] if ends else rawd
        cs, sn, rows = cd[gone:], sd[gone:], most - gone
        masks = []
        for path in ("own calls", "one call", "one launch"):
            own = keys.clone()
            sc = torch.full((1, cols), -7.0, dtype=torch.float32, device="cuda")
            mask = torch.full((1, most - gone), 0xAB, dtype=torch.uint8, device="cuda")
            st = qsa.new_status()
            if path == "own calls":
                if ends:
                    qsa.qsa_pool_blocks(block_raw, 128, block, 1, kwd, cs, sn, rows, EPS, own)
                qsa.qsa_score_rows(q, 640, dev(np.array([true], np.int32)), dev(np.array([at + 1], np.int32)), 1, most, qwd, cd,
                                   sd, most, EPS, own, None, sc, cols, st)
                qsa.qsa_select_mask(sc, cols, dev(np.array([at], np.int32)), 1, most - gone, select, mask, st)
            else:
                args = (block_raw, 128, block if ends else 0, int(ends), kwd, q, 640, dev(np.array([at], np.int32)), 1, most - gone,
                        qwd, cs, sn, rows, EPS, select, own, sc, cols, mask, st)
                if path == "one call":
                    qsa.qsa_index_select(*args)
                else:
                    qsa.qsa_decode_index_select(*args, ws)
            assert qsa.qsa_read_status(st) == (0, 0), path
            assert np.array_equal(own[:seen].cpu().numpy().view(np.uint16), want_keys), path
            got = sc.cpu().numpy()
            want = np.full((1, cols), -7.0, np.float32)
            rc, _ = orc.score_rows(fq[i:i + 1], 640, np.array([true], np.int32), 1, most, qw, cos_t, sin_t, EPS,
                                   np.ascontiguousarray(want_keys), want, cols, visible_len=np.array([at + 1], np.int32))
            assert rc == 0
            assert_close(got[0, :seen], want[0, :seen], path)
            expect, rc = orc.select_row(got[0], at, most - gone, select)
            assert rc == 0 and np.array_equal(mask.cpu().numpy()[0], expect), path
            masks.append(mask)
            stepped = own
        keys = stepped
        # what the row attends: the selected tokens' K and V, and the attention over them
        cap = select + 3
        chosen = torch.full((1, cap), -1, dtype=torch.int32, device="cuda")
        count = torch.zeros(1, dtype=torch.int32, device="cuda")
        qsa.qsa_mask_tokens(masks[-1], 1, most - gone, chosen, cap, count)
        n = int(count.item())
        picked = chosen.cpu().numpy()[0, :n]
        assert np.array_equal(picked, np.nonzero(masks[-1].cpu().numpy()[0])[0])
        places = np.asarray(tokens, int)[picked]
        ko, vo = (torch.zeros((cap, width), dtype=torch.int16, device="cuda") for _ in range(2))
        st = qsa.new_status()
        qsa.qsa_gather_kv(kd, vd, width, pages, td, pages, pages, page, chosen, cap, count, 1, cap, ko, vo, cap, st)
        assert np.array_equal(ko[:n].cpu().numpy().view(np.uint16), k[places])
        assert np.array_equal(vo[:n].cpu().numpy().view(np.uint16), v[places])
        qa = qi.normal_bf16(rng, (1, row), 1.5)
        out = torch.zeros((1, row), dtype=torch.int16, device="cuda")
        qsa.qsa_sparse_attn(dev(qa), row, nq, nkv, hd, kd, vd, pages, page, td, pages, pages, chosen, cap, count, 1, cap, scale,
                            out, row, st)
        assert qsa.qsa_read_status(st) == (0, 0)
        # each weight is rounded once, in the sum over V and in the normaliser alike
        qf, kf, vf = f64(qa).reshape(nq, hd), f64(k[places]).reshape(n, nkv, hd), f64(v[places]).reshape(n, nkv, hd)
        for h in range(nq):
            s = kf[:, h // 4] @ qf[h] * scale
            delta = scale * (hd + 4) * 2 * U * float((np.abs(kf[:, h // 4]) @ np.abs(qf[h])).max())
            p = np.exp(s - s.max())
            p /= p.sum()
            tol = (2 * BF + 4 * delta + 2 ** -20 + 4 * n * U) * (p @ np.abs(vf[:, h // 4]))
            y = p @ vf[:, h // 4]
            assert np.all(np.abs(f64(out.cpu().numpy().view(np.uint16)[0, h * hd:(h + 1) * hd]) - y) <= tol + BF * np.abs(y))
