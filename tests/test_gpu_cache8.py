"""qsa_cache8_attn against the plain form in 64 bits (step_cases.ref_attend; the
tolerances are derived there)."""
import threading

import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev, f64
from step_cases import Cache8, ref_attend

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
        ws = qsa.new_cache8_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd)
        ws.fill_(0xFF)  # NaNs: its contents do not matter
    args = c.args(dev(qb), row + q_pad)
    torch.cuda.synchronize()
    qsa.qsa_cache8_attn(*args, c.hd ** -0.5 if scale is None else scale, out, row + out_pad, l, st, ws, stream=stream)
    torch.cuda.synchronize()
    o = out.cpu().numpy().view(np.uint16)
    assert np.all(o[:, row:] == SENT), "wrote past a row"
    return o[:, :row], None if l is None else l.cpu().numpy(), qsa.qsa_read_status(st)


def check(c, out, lse, scale=None, seqs=None):
    scale = c.hd ** -0.5 if scale is None else scale
    owned = np.zeros(c.n_rows, bool)
    worst = 0.0
    for i in range(c.n) if seqs is None else seqs:
        want, tol, wl, ltol = ref_attend(c, i, scale)
        r0, m = int(c.row_start[i]), int(c.rows[i])
        owned[r0:r0 + m] = True
        got = f64(out[r0:r0 + m]).reshape(m, c.nq, c.hd)
        assert np.array_equal(np.isnan(got), np.isnan(want)), f"sequence {i}: NaN pattern"
        fin = np.isfinite(want)
        err = np.abs(got[fin] - want[fin])
        worst = max(worst, float(np.max(err / np.maximum(tol[fin], 1e-300), initial=0.0)))
        assert np.all(err <= tol[fin]), f"sequence {i}: {np.max(err / tol[fin])} of the bound"
        gl = lse[r0:r0 + m]
        assert np.array_equal(np.isneginf(gl), np.isneginf(wl)) and np.array_equal(np.isnan(gl), np.isnan(wl))
        ok = np.isfinite(wl)
        assert np.all(np.abs(gl[ok] - wl[ok]) <= ltol[ok]), np.max(np.abs(gl[ok] - wl[ok]) / ltol[ok])
    if seqs is None:
        assert np.all(out[~owned] == SENT), "a row outside every sequence was written"
        assert np.all(lse[~owned] == 123.0)
    return worst


SHAPES = [(16, 2, 256, 16, 16), (8, 1, 128, 32, 16), (32, 8, 128, 64, 64), (24, 2, 256, 128, 128), (6, 2, 128, 96, 32),
          (4, 4, 256, 64, 16)]


@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
@pytest.mark.parametrize("nq,nkv,hd,page,unit", SHAPES)
def test_ragged_batch(qsa, nq, nkv, hd, page, unit, mask):
    """Contexts of 0, 1 and around the tile's 128 tokens, sequences without rows, with
    one, and with more than 32 drafted tokens; rows outside every sequence."""
    rng = qi.rng_for(70, salt=nq * 100 + hd + page)
    c = Cache8(rng, [0, 1, 127, 128, 129, 300, 90, 255], [3, 1, 1, 5, 0, 40, 38, 2], nq, nkv, hd, page, unit, mask, gaps=2)
    out, lse, st = call(qsa, c, q_pad=8, out_pad=16)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("nq,nkv,hd", [(16, 2, 256), (32, 8, 128), (40, 2, 128), (2, 2, 256), (128, 1, 128)])
def test_single_tokens(qsa, nq, nkv, hd):
    """Every width of a KV head's group, to more heads than a tile has rows."""
    rng = qi.rng_for(71, salt=hd + nq)
    c = Cache8(rng, [0, 1, 63, 511, 514, 1000], [1] * 6, nq, nkv, hd, 16, 16, "chain")
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)
    nolse, none, st = call(qsa, c, lse=False)
    assert st == (0, 0) and np.array_equal(nolse, out)


@pytest.mark.parametrize("rows,mask", [(4, "tree"), (9, "chain"), (70, "tree"), (129, "tree"), (300, "chain"), (200, "random")])
@pytest.mark.parametrize("hd", [128, 256])
def test_wide_trees_and_chunks(qsa, hd, rows, mask):
    """More rows than one tile of the products holds, group 3 (no power of two)."""
    rng = qi.rng_for(72, salt=rows + hd)
    c = Cache8(rng, [77, 0], [rows, 9], 6, 2, hd, 16, 16, mask)
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("hd,nq,nkv", [(256, 16, 2), (128, 8, 8)])
def test_long_context_beside_short_ones(qsa, hd, nq, nkv):
    """One context that many CTAs share, among ones that a CTA has whole."""
    rng = qi.rng_for(73, salt=hd)
    c = Cache8(rng, [12, 20011, 700, 4096], [2, 4, 1, 3], nq, nkv, hd, 16, 16, "tree")
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("n", [33, 700])
def test_many_sequences(qsa, n):
    rng = qi.rng_for(74, salt=n)
    c = Cache8(rng, rng.integers(0, 150, n), rng.integers(0, 4, n), 8, 2, 128, 32, 32, "tree")
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("n_first,window", [(0, 1), (0, 7), (4, 100), (16, 128), (130, 129), (1, 1000), (300, 40), (0, 2 ** 31 - 1),
                                            (2 ** 31 - 1, 1)])
@pytest.mark.parametrize("mask", ["chain", "tree"])
def test_windows(qsa, n_first, window, mask):
    """First tokens and the window's edge inside, at and past a tile's ends; windows shorter than the drafted rows."""
    rng = qi.rng_for(75, salt=window % 1000 + n_first % 1000)
    for nq, nkv, hd, rows in ((16, 2, 256, [1] * 6), (8, 2, 128, [37, 1, 5, 70, 0, 12])):
        c = Cache8(rng, [0, 1, 129, 400, 1100, 515], rows, nq, nkv, hd, 32, 32, mask, n_first=n_first, window=window)
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)


def test_window_over_a_long_context(qsa):
    """A window in a long cache: pages that no row sees may be anything, a table entry outside the pool among them."""
    rng = qi.rng_for(76)
    for rows, mask in ([1, 1], "chain"), ([20, 3], "tree"), ([300, 2], "chain"):
        c = Cache8(rng, [9000, 5000], rows, 16, 2, 256, 16, 16, mask, n_first=20, window=700)
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)
        c.table[0, 100:500] = -5
        again, lse2, st = call(qsa, c)
        assert st == (0, 0) and np.array_equal(again, out) and np.array_equal(lse2, lse)


def test_rows_that_see_nothing(qsa):
    rng = qi.rng_for(77)
    c = Cache8(rng, [0, 0, 5], [4, 1, 3], 16, 2, 256, 16, 16, "tree")
    c.set_bits(0, np.array([[0, 0, 0, 0], [1, 0, 0, 0], [0, 0, 0, 0], [1, 1, 0, 0]], bool))
    c.set_bits(1, np.zeros((1, 1), bool))
    c.set_bits(2, np.zeros((3, 3), bool))
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)
    for r in (0, 2, 4):
        assert np.all(out[r] == 0) and np.all(np.isneginf(lse[r]))


@pytest.mark.parametrize("hd", [128, 256])
def test_nan_stays_with_the_rows_that_see_it(qsa, hd):
    """NaN in drafted K and V rows, in tokens outside a window, and in every slot past the sequences' tokens."""
    rng = qi.rng_for(78, salt=hd)
    for mask, n_first, window in (("tree", 0, 0), ("chain", 0, 0), ("tree", 8, 60), ("chain", 3, 9)):
        c = Cache8(rng, [100, 0, 250], [20, 6, 12], 8, 2, hd, 16, 16, mask, n_first=n_first, window=window)
        used = np.concatenate([c.slots(i, np.arange(c.ctx[i] + c.rows[i])) for i in range(c.n)])
        past = np.setdiff1d(np.arange(c.k.shape[0]), used)
        clean, clean_lse, _ = call(qsa, c)
        c.k[past], c.v[past] = 0x7F, 0xFF
        out, lse, st = call(qsa, c)
        assert st == (0, 0) and np.array_equal(out, clean) and np.array_equal(lse, clean_lse)
        # a V value and a K row of drafted tokens, a V value of a context token
        c.v[c.slots(0, 105), 1, 3] = 0x7F
        c.v[c.slots(0, 119), 0, hd - 1] = 0xFF
        c.k[c.slots(2, 255), 0, 9] = 0x7F
        c.v[c.slots(2, 240), 1, 77] = 0x7F
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)


def test_scales_far_apart(qsa):
    """Blocks of V and K whose scales differ by much, zero ones among them, where little or much weight lies on them."""
    rng = qi.rng_for(79)
    for trial in range(4):
        c = Cache8(rng, [700, 40], [3, 1], 16, 2, 256, 16, 16, "tree")
        c.vs = (c.vs * np.exp2(rng.integers(-24, 24, c.vs.shape) * (trial % 2 + 0.25))).astype(np.float32)
        c.ks = (c.ks * np.exp2(rng.integers(-3, 3, c.ks.shape))).astype(np.float32)
        if trial > 1:
            c.vs[rng.random(c.vs.shape) < 0.4] = 0
            c.ks[rng.random(c.ks.shape) < 0.3] = 0
        out, lse, st = call(qsa, c)
        assert st == (0, 0)
        check(c, out, lse)
    c.vs[:] = 0
    out, lse, st = call(qsa, c)
    assert st == (0, 0) and np.all(f64(out) == 0)
    check(c, out, lse)


def test_a_key_far_above_the_others(qsa):
    """The largest logit late, early and at the edges of tiles: references move by little and by much."""
    rng = qi.rng_for(80)
    for hd, nq, nkv in ((256, 16, 2), (128, 6, 2)):
        for at in (0, 1, 127, 128, 255, 256, 383, 640, 899):
            c = Cache8(rng, [890], [10], nq, nkv, hd, 16, 16, "tree" if at < 890 else "chain", q_std=3.0)
            c.ks[int(c.slots(0, at)) // 16] *= 16
            out, lse, st = call(qsa, c)
            assert st == (0, 0)
            check(c, out, lse)


def test_logits_that_grow(qsa):
    """Every tile's largest logit above the one before: the reference moves in each."""
    rng = qi.rng_for(81)
    c = Cache8(rng, [2000], [4], 8, 2, 128, 16, 16, "tree")
    for t in range(0, 2000, 16):
        c.ks[int(c.slots(0, t)) // 16] *= np.float32(1 + t / 100)
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.0625, 1.0, 1e-30])
def test_scales_of_logits(qsa, scale):
    rng = qi.rng_for(82)
    for hd in (128, 256):
        c = Cache8(rng, [300, 5], [4, 1], 8, 2, hd, 16, 16, "tree")
        out, lse, st = call(qsa, c, scale=scale)
        assert st == (0, 0)
        check(c, out, lse, scale=scale)


def test_queries_of_every_size(qsa):
    """Heads of zeros, of one large value among small ones, of tiny and of huge values."""
    rng = qi.rng_for(83)
    c = Cache8(rng, [300], [6], 8, 2, 128, 16, 16, "tree")
    q = f64(c.q).reshape(6, 8, 128)
    q[0] = 0
    q[1, :, 5] *= 1000
    q[2] *= 2.0 ** -80
    q[3] *= 2.0 ** 30
    q[4] *= 2.0 ** np.arange(-16, 0).repeat(8)[None]
    c.q = qi.to_bf16_bits(q.reshape(6, -1).astype(np.float32))
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse)


def test_repeats_its_bits(qsa):
    rng = qi.rng_for(84)
    c = Cache8(rng, [3000, 77, 1200], [5, 40, 1], 16, 2, 256, 16, 16, "tree")
    out, lse, _ = call(qsa, c)
    for _ in range(3):
        o, l, st = call(qsa, c)
        assert st == (0, 0) and np.array_equal(o, out) and np.array_equal(l, lse)


def test_bad_sequences_alone(qsa):
    rng = qi.rng_for(85)
    base = Cache8(rng, [300, 100, 40, 700], [5, 3, 9, 2], 16, 2, 256, 16, 16, "tree")
    out, lse, st = call(qsa, base)
    assert st == (0, 0)
    r = base.row_start
    for what in range(5):
        c = base
        ctx, start, words = c.ctx.copy(), c.row_start.copy(), c.words
        if what == 0:
            c.ctx[1] = -4
        elif what == 1:
            c.ctx[1] = c.table_len * 16 - 2
        elif what == 2:
            c.ctx[1] = 2 ** 31 - 1
        elif what == 3:
            c.row_start[1] = c.n_rows + 9  # the first and the second are bad
        else:
            c.row_start[1] = -1
        o, l, st = call(qsa, c)
        assert st[0] == 3 and st[1] in (0, 1)
        first = int(r[2]) if what >= 3 else int(r[1])
        if what < 3:
            assert np.array_equal(o[:first], out[:first]) and np.array_equal(l[:first], lse[:first])
        assert np.all(o[int(r[1]):int(r[2])] == SENT)
        a, b = f64(o[int(r[2]):]), f64(out[int(r[2]):])
        assert np.allclose(a, b, rtol=2.0 ** -6, atol=2.0 ** -6)  # another split of the work
        c.ctx, c.row_start, c.words = ctx, start, words


def test_bad_pages_and_scales(qsa):
    rng = qi.rng_for(86)
    c = Cache8(rng, [300, 100], [5, 3], 16, 2, 256, 16, 16, "tree")
    out, lse, _ = call(qsa, c)
    keep = c.table[1, 2]
    for bad in (-1, c.pages, 2 ** 31 - 1):
        c.table[1, 2] = bad
        o, l, st = call(qsa, c)
        assert st == (6, 1)
    c.table[1, 2] = keep
    for arr in (c.ks, c.vs):
        blk = int(c.slots(1, 50)) // 16
        was = arr[blk, 1]
        for bad in (-1.0, np.nan, np.inf):
            arr[blk, 1] = bad
            o, l, st = call(qsa, c)
            assert st == (4, 1), bad
            assert np.allclose(f64(o[:5]), f64(out[:5]), rtol=2.0 ** -6, atol=2.0 ** -6)
        arr[blk, 1] = was


def test_streams_graphs_and_shared_workspace(qsa):
    """Two captured calls of different shapes over one workspace, replayed in turn; two threads on their own streams."""
    rng = qi.rng_for(87)
    cases = [Cache8(rng, [3000, 77], [5, 40], 16, 2, 256, 16, 16, "tree"), Cache8(rng, [40, 900, 60], [1, 1, 1], 16, 2, 256, 32, 16, "chain")]
    want = [call(qsa, c) for c in cases]
    ws = qsa.new_cache8_workspace(3, 45, 16, 2, 256)
    side = torch.cuda.Stream()
    made = []
    for c in cases:
        q = dev(c.q)
        out = torch.zeros(c.q.shape, dtype=torch.int16, device="cuda")
        lse = torch.zeros((c.n_rows, c.nq), dtype=torch.float32, device="cuda")
        st, d = qsa.new_status(), c.device()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            qsa.qsa_cache8_attn(*c.args(q, 16 * 256, d), 0.0625, out, 16 * 256, lse, st, ws)
        made.append((g, q, out, lse, st, d))
    for k in range(6):
        made[k % 2][0].replay()
    torch.cuda.synchronize()
    for (_, _, out, lse, st, _), (o, l, _) in zip(made, want):
        assert np.array_equal(out.cpu().numpy().view(np.uint16), o) and np.array_equal(lse.cpu().numpy(), l)
        assert qsa.qsa_read_status(st) == (0, 0)
    got = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = call(qsa, cases[i])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
