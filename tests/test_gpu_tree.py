"""qsa_tree_attn against the plain form in 64 bits (cache_cases.ref_tree; the
tolerances are derived there)."""
import threading

import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev, f64, ref_tree

pytestmark = pytest.mark.gpu
SENT = 0x7FAB


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def call(qsa, c, scale=None, q_pad=0, out_pad=0, lse=True, stream=None, ws=None):
    """One call; returns out bits [n_rows, nq*hd], lse [n_rows, nq], status."""
    row = c.nq * c.hd
    qb = np.zeros((c.n_rows, row + q_pad), np.uint16)
    qb[:, :row] = c.q
    out = torch.full((c.n_rows, row + out_pad), SENT, dtype=torch.int16, device="cuda")
    l = torch.full((c.n_rows, c.nq), 123.0, dtype=torch.float32, device="cuda") if lse else None
    st = qsa.new_status()
    if ws is None:
        ws = qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd)
        ws.fill_(0xFF)  # NaNs: its contents do not matter
    args = c.tree_args(dev(qb), row + q_pad)
    torch.cuda.synchronize()
    qsa.qsa_tree_attn(*args, c.hd ** -0.5 if scale is None else scale, out, row + out_pad, l, st, ws, stream=stream)
    torch.cuda.synchronize()
    o = out.cpu().numpy().view(np.uint16)
    assert np.all(o[:, row:] == SENT), "wrote past a row"
    return o[:, :row], None if l is None else l.cpu().numpy(), qsa.qsa_read_status(st)


def check(c, out, lse, scale=None, seqs=None, rows=None):
    scale = c.hd ** -0.5 if scale is None else scale
    owned = np.zeros(c.n_rows, bool)
    for i in range(c.n) if seqs is None else seqs:
        want, tol, wl, ltol = ref_tree(c, i, scale)
        r0, m = int(c.row_start[i]), int(c.rows[i])
        owned[r0:r0 + m] = True
        got = f64(out[r0:r0 + m]).reshape(m, c.nq, c.hd)
        assert np.array_equal(np.isnan(got), np.isnan(want)), f"sequence {i}: NaN pattern"
        fin = np.isfinite(want)
        assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
        err = np.abs(got - want)[fin]
        assert np.all(err <= tol[fin]), f"sequence {i}: {np.max(err / tol[fin])} of the bound"
        if lse is not None:
            gl = lse[r0:r0 + m]
            assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
            ok = np.isfinite(wl)
            assert np.array_equal(np.isnan(gl), np.isnan(wl))
            assert np.all(np.abs(gl - wl)[ok] <= ltol[ok]), np.max((np.abs(gl - wl) / ltol)[ok])
    if seqs is None:
        assert np.all(out[~owned] == SENT), "a row outside every sequence was written"
        if lse is not None:
            assert np.all(lse[~owned] == 123.0)


@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
@pytest.mark.parametrize("nq,nkv,hd,page", [(16, 2, 256, 16), (8, 1, 128, 7), (6, 2, 128, 64), (24, 2, 256, 1),
                                            (4, 4, 256, 100), (32, 8, 128, 16)])
def test_ragged_batch(qsa, nq, nkv, hd, page, mask):
    """Contexts of 0, 1 and around the tile's 128 tokens, sequences without rows, with
    one, and with more than 32 drafted tokens; rows outside every sequence."""
    rng = qi.rng_for(20, salt=nq * 100 + hd + page)
    c = Cache(rng, [0, 1, 127, 128, 129, 300, 90, 255], [3, 1, 1, 5, 0, 40, 38, 2], nq, nkv, hd, page, mask, gaps=2)
    out, lse, st = call(qsa, c, q_pad=8, out_pad=16)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("nq,nkv,hd", [(16, 2, 256), (32, 8, 128)])
def test_single_tokens(qsa, nq, nkv, hd):
    rng = qi.rng_for(21, salt=hd)
    c = Cache(rng, [0, 1, 63, 511, 514, 1000], [1] * 6, nq, nkv, hd, 16, "chain")
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)
    nolse, none, st = call(qsa, c, lse=False)
    assert st == (0, 0) and np.array_equal(nolse, out)


@pytest.mark.parametrize("rows,mask", [(70, "tree"), (129, "tree"), (300, "chain"), (200, "random")])
@pytest.mark.parametrize("hd", [128, 256])
def test_wide_trees_and_chunks(qsa, hd, rows, mask):
    """More rows than one tile of the products holds, group 3 (no power of two)."""
    rng = qi.rng_for(22, salt=rows + hd)
    c = Cache(rng, [77, 0], [rows, 9], 6, 2, hd, 16, mask)
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("hd,nq,nkv", [(256, 16, 2), (128, 8, 8)])
def test_long_context_beside_short_ones(qsa, hd, nq, nkv):
    """One context that many CTAs share, among ones that a CTA has whole."""
    rng = qi.rng_for(23, salt=hd)
    c = Cache(rng, [12, 20011, 700, 4096], [2, 4, 1, 3], nq, nkv, hd, 16, "tree")
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


def test_rows_that_see_nothing(qsa):
    rng = qi.rng_for(24)
    c = Cache(rng, [0, 0, 5], [4, 1, 3], 16, 2, 256, 16, "tree")
    c.set_bits(0, np.array([[0, 0, 0, 0], [1, 0, 0, 0], [0, 0, 0, 0], [1, 1, 0, 0]], bool))
    c.set_bits(1, np.zeros((1, 1), bool))
    c.set_bits(2, np.zeros((3, 3), bool))
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)
    for r in (0, 2, 4):
        assert np.all(out[r] == 0) and np.all(np.isneginf(lse[r]))


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_nonfinite_values_stay_with_the_rows_that_see_them(qsa, hd, bad):
    """Drafted K and V rows with NaN or infinities, and every slot past the
    sequences' tokens: only rows whose mask names such a token show it."""
    rng = qi.rng_for(25, salt=hd)
    c = Cache(rng, [100, 0, 250], [20, 6, 12], 8, 2, hd, 16, "tree")
    word = qi.to_bf16_bits(np.array([bad], np.float32))[0]
    used = np.concatenate([c.slots(i, np.arange(c.ctx[i] + c.rows[i])) for i in range(c.n)])
    past = np.setdiff1d(np.arange(c.k.shape[0]), used)
    clean, clean_lse, _ = call(qsa, c)
    c.k[past] = word
    c.v[past] = word
    out, lse, st = call(qsa, c)
    assert st == (0, 0) and np.array_equal(out, clean) and np.array_equal(lse, clean_lse)
    # drafted token 3 of sequence 0 and 2 of sequence 2: one value, one whole row
    s0, s2 = c.slots(0, [103])[0], c.slots(2, [252])[0]
    c.v[s0, 5] = word
    c.v[s2, hd:] = word   # KV head 1
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)
    blind = [j for j in range(20) if not c.sees(0)[j, 3]]
    assert blind and np.array_equal(out[blind], clean[blind])
    # a key of which only the seeing rows may know
    c.k[s0, :] = word
    out, lse, st = call(qsa, c)
    assert st == (0, 0) and np.array_equal(out[blind], clean[blind]) and np.array_equal(lse[blind], clean_lse[blind])
    seeing = [j for j in range(20) if c.sees(0)[j, 3]]
    assert seeing and not np.any(np.isfinite(f64(out[seeing]).reshape(len(seeing), 8, hd)[..., 5]))


def test_dominant_tokens(qsa):
    """Each row's own drafted token, or one context token, has nearly all the weight:
    a wrong token, page or head is an error of order one."""
    rng = qi.rng_for(26)
    c = Cache(rng, [700, 41], [5, 33], 8, 2, 128, 7, "tree", q_std=1.0)
    for i in range(c.n):
        for j in range(int(c.rows[i])):
            t = int(rng.integers(0, c.ctx[i])) if j % 2 else int(c.ctx[i]) + j
            for g in range(c.nkv):
                row = c.q[c.row_start[i] + j].reshape(c.nq, c.hd)
                c.k[c.slots(i, [t])[0]].reshape(c.nkv, c.hd)[g] = qi.to_bf16_bits(
                    (4 * qi.bf16_bits_to_f32(row[g * c.group])).astype(np.float32))
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


def test_large_logits_and_growing_maxima(qsa):
    """Logits of hundreds whose running maximum grows along the context."""
    rng = qi.rng_for(27)
    c = Cache(rng, [1500], [3], 16, 2, 256, 16, "chain", q_std=1.0)
    for t in range(1500):
        s = c.slots(0, [t])[0]
        c.k[s] = qi.to_bf16_bits(qi.bf16_bits_to_f32(c.k[s]) * np.float32(0.1 + t / 50))
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


def test_shared_prefix_pages_and_one_table(qsa):
    """Sequences whose tables name the same pages, and table_cols 0."""
    rng = qi.rng_for(28)
    c = Cache(rng, [200, 200], [3, 3], 8, 2, 128, 16, "chain")
    c.table[1] = c.table[0]
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)
    d = c.device()
    o2 = torch.zeros((c.n_rows, c.nq * c.hd), dtype=torch.int16, device="cuda")
    s2 = qsa.new_status()
    qsa.qsa_tree_attn(dev(c.q), c.nq * c.hd, c.nq, c.nkv, c.hd, d["k"], d["v"], c.pages, c.page, dev(c.table[0]),
                      c.table_len, 0, d["ctx"], d["start"], c.n, c.n_rows, None, 0, c.hd ** -0.5, o2, c.nq * c.hd, None, s2,
                      qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd))
    assert qsa.qsa_read_status(s2) == (0, 0)
    assert np.array_equal(o2.cpu().numpy().view(np.uint16), out)


def test_device_errors_leave_the_other_sequences(qsa):
    rng = qi.rng_for(29)
    for kind in ("context", "negative", "rows", "mask", "page"):
        c = Cache(rng, [50, 60, 70], [4, 40, 4], 8, 2, 128, 16, "tree")
        good, glse, st = call(qsa, c)
        assert st == (0, 0)
        want = (3, 1)
        if kind == "context":
            c.ctx[1] = c.table_len * 16 - 39
        elif kind == "negative":
            c.ctx[1] = -1
        elif kind == "rows":
            c.row_start[1:] = [4, 49, 48]   # sequence 1 runs past n_rows, sequence 2 backwards
            want = None
        elif kind == "mask":
            c.mask = np.ascontiguousarray(c.mask[:, :1])
            c.words = 1
        else:
            c.table[1, 2] = c.pages
            want = (6, 1)
        if kind == "page":
            out, lse, st = call(qsa, c)
        else:
            out, lse, st = call(qsa, c)
            assert np.all(out[4:44] == SENT) and np.all(lse[4:44] == 123.0)
        assert st == want if want else (st[0] == 3 and st[1] in (1, 2))
        r = [0, 1, 2, 3] if kind == "rows" else [0, 1, 2, 3, 44, 45, 46, 47]
        assert np.array_equal(out[r], good[r]) and np.array_equal(lse[r], glse[r])


def test_repeats_graphs_and_streams(qsa):
    """The same bits again, on another stream, and from a graph whose inputs change."""
    rng = qi.rng_for(30)
    c = Cache(rng, [3000, 9, 500], [7, 2, 30], 16, 2, 256, 16, "tree")
    out, lse, st = call(qsa, c)
    ws = qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd)
    for stream in (None, torch.cuda.Stream()):
        o, l, st = call(qsa, c, stream=stream, ws=ws)
        assert st == (0, 0) and np.array_equal(o, out) and np.array_equal(l, lse)
    row = c.nq * c.hd
    q = dev(c.q)
    ctx = dev(c.ctx)
    args = list(c.tree_args(q, row))
    args[12] = ctx
    o = torch.zeros((c.n_rows, row), dtype=torch.int16, device="cuda")
    l = torch.zeros((c.n_rows, c.nq), dtype=torch.float32, device="cuda")
    stat = qsa.new_status()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        qsa.qsa_tree_attn(*args, c.hd ** -0.5, o, row, l, stat, ws)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(o.cpu().numpy().view(np.uint16), out) and np.array_equal(l.cpu().numpy(), lse)
    shorter = Cache.__new__(Cache)
    shorter.__dict__ = dict(c.__dict__, ctx=np.array([2000, 3, 400], np.int32))
    ctx.copy_(dev(shorter.ctx))
    g.replay()
    torch.cuda.synchronize()
    check(shorter, o.cpu().numpy().view(np.uint16), l.cpu().numpy())
    assert qsa.qsa_read_status(stat) == (0, 0)


def test_two_host_threads(qsa):
    cs = [Cache(qi.rng_for(31, salt=i), [900, 40], [5, 17], 8, 2, 128 * (i + 1), 16, "tree") for i in range(2)]
    want = [call(qsa, c) for c in cs]
    got, errors, gate = [None, None], [], threading.Barrier(2)

    def worker(i):
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            gate.wait()
            for _ in range(10):
                got[i] = call(qsa, cs[i], stream=st)
        except Exception as e:
            errors.append(repr(e))

    ts = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    for g, w in zip(got, want):
        assert g[2] == (0, 0) and np.array_equal(g[0], w[0]) and np.array_equal(g[1], w[1])


def test_agrees_with_sparse_attention_over_every_token(qsa):
    """One decode row over the whole cache equals qsa_sparse_attn given every token."""
    rng = qi.rng_for(32)
    c = Cache(rng, [640], [1], 16, 2, 256, 16, "chain")
    out, _, st = call(qsa, c)
    assert st == (0, 0)
    d = c.device()
    sel = torch.arange(641, dtype=torch.int32, device="cuda").view(1, -1)
    o = torch.zeros((1, c.nq * c.hd), dtype=torch.int16, device="cuda")
    s = qsa.new_status()
    qsa.qsa_sparse_attn(dev(c.q), c.nq * c.hd, c.nq, c.nkv, c.hd, d["k"], d["v"], c.pages, c.page, d["table"],
                        c.table_len, 0, sel, 641, torch.tensor([641], dtype=torch.int32, device="cuda"), 1, 641,
                        c.hd ** -0.5, o, c.nq * c.hd, s)
    assert qsa.qsa_read_status(s) == (0, 0)
    _, tol, _, _ = ref_tree(c, 0, c.hd ** -0.5)
    assert np.all(np.abs(f64(o.cpu().numpy().view(np.uint16)) - f64(out)) <= 2 * tol.reshape(1, -1))
