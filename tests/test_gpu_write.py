"""qsa_qkv_write against the plain form in 64 bits (step_cases; tolerances derived there)."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import BF, U, dev, f64
from step_cases import E4M3, pool_8, ref_heads, scale_of, to_e4m3

pytestmark = pytest.mark.gpu
SENT = 0x7FAB


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


class Write:
    """n sequences, their new rows' q, k and v (one projection's rows), and a cache of 8 or 16 bits."""

    def __init__(self, qsa, rng, ctx, rows, nq, nkv, hd, page, unit=16, bits=8, gaps=0, norm=True, pos=None, table_rows=None):
        self.ctx, self.rows = np.asarray(ctx, np.int32), np.asarray(rows, np.int32)
        self.nq, self.nkv, self.hd, self.page, self.unit, self.bits, self.n = nq, nkv, hd, page, unit, bits, len(ctx)
        per = np.maximum(1, -(-(self.ctx + self.rows) // page))
        self.table_len, self.pages = int(per.max()), int(per.sum()) + 2
        order = rng.permutation(self.pages)
        self.table = np.full((self.n, self.table_len), -1, np.int32)
        at = 0
        for i, p in enumerate(per):
            self.table[i, :p] = order[at:at + p]
            at += int(p)
        self.row_start = (np.concatenate([[0], np.cumsum(self.rows)]) + gaps).astype(np.int32)
        self.n_rows = int(self.row_start[-1]) + gaps
        self.x = qi.normal_bf16(rng, (self.n_rows, (nq + 2 * nkv) * hd + 8), std=2.0)
        self.qw, self.kw = (qi.normal_bf16(rng, (hd,), 0.1) for _ in range(2)) if norm else (None, None)
        self.eps, self.pos = 1e-6, pos
        self.table_rows = int((self.ctx + self.rows).max()) if table_rows is None else table_rows
        self.cos, self.sin = qsa.qsa_rope_tables(self.table_rows, 10000.0)
        tokens = self.pages * page
        if bits == 8:
            (self.k, self.ks), (self.v, self.vs) = (pool_8(rng, tokens, nkv, hd, unit) for _ in range(2))
        else:
            self.k, self.v = (qi.normal_bf16(rng, (tokens, nkv, hd)) for _ in range(2))
            self.ks = self.vs = None

    def slots(self, i, t):
        t = np.asarray(t)
        return self.table[i, t // self.page].astype(np.int64) * self.page + t % self.page

    def run(self, qsa, inplace=False, stream=None, capture=False):
        nq, nkv, hd = self.nq, self.nkv, self.hd
        d = nq * hd
        x, stride = dev(self.x), self.x.shape[1]
        q, k, v = x[:, :d], x[:, d:d + nkv * hd], x[:, d + nkv * hd:]
        out = x if inplace else torch.full((self.n_rows, d + 16), SENT, dtype=torch.int16, device="cuda")
        opt = lambda a: None if a is None else dev(a)  # noqa: E731
        pools = [opt(a) for a in (self.k, self.v, self.ks, self.vs)]
        st = qsa.new_status()
        args = (q, stride, nq, k, stride, v, stride, nkv, hd, opt(self.qw), opt(self.kw), self.eps, dev(self.cos), dev(self.sin),
                self.table_rows, opt(self.pos), dev(self.ctx), dev(self.row_start), self.n, self.n_rows, *pools, self.unit,
                self.pages, self.page, dev(self.table), self.table_len, self.table_len, out, out.shape[1], st)
        torch.cuda.synchronize()
        qsa.qsa_qkv_write(*args, stream=stream)
        torch.cuda.synchronize()
        o = out.cpu().numpy().view(np.uint16)
        if not inplace:
            assert np.all(o[:, d:] == SENT)
        got = [None if p is None else p.cpu().numpy() for p in pools]
        if self.bits == 16:
            got[:2] = [g.view(np.uint16) for g in got[:2]]
        return o[:, :d], got, qsa.qsa_read_status(st)

    def check(self, o, got, left_alone=(), untouched=None):
        """left_alone: rows whose position is out of range."""
        nq, nkv, hd, u = self.nq, self.nkv, self.hd, self.unit
        d = nq * hd
        x = f64(self.x)
        owned = np.zeros(self.n_rows, bool)
        pools = [a if a is None else a.copy() for a in (self.k, self.v, self.ks, self.vs)]
        touched = np.zeros(self.pages * self.page, bool)
        for i in range(self.n):
            m, c, r0 = int(self.rows[i]), int(self.ctx[i]), int(self.row_start[i])
            keep = np.array([j for j in range(m) if r0 + j not in left_alone], int)
            rows, tok = r0 + keep, c + keep
            owned[rows] = True
            if len(keep) == 0:
                continue
            at = tok if self.pos is None else self.pos[rows]
            cos, sin = f64(self.cos[at]), f64(self.sin[at])
            w = [None if a is None else f64(a) for a in (self.qw, self.kw)]
            want, tol = ref_heads(x[rows, :d].reshape(-1, nq, hd), w[0], self.eps, cos, sin)
            y = f64(o[rows]).reshape(-1, nq, hd)
            assert np.all(np.abs(y - want) <= tol + BF * np.abs(want) + 1e-30), f"sequence {i}: q"
            slots = self.slots(i, tok)
            touched[slots] = True
            for which in (0, 1):
                lo = d + which * nkv * hd
                raw = x[rows, lo:lo + nkv * hd].reshape(-1, nkv, hd)
                want, tol = ref_heads(raw, w[1], self.eps, cos, sin) if which == 0 else (raw, np.zeros_like(raw))
                if self.bits == 16:
                    y = f64(got[which][slots])
                    assert np.all(np.abs(y - want) <= tol + BF * np.abs(want) + 1e-30), f"sequence {i}: pool {which}"
                    continue
                for b in range(c // u, (c + m - 1) // u + 1):
                    mine = tok // u == b
                    if not mine.any():
                        continue
                    blk = int(self.slots(i, b * u)) // u
                    amax = np.abs(want[mine]).max((0, 2))
                    edge = tol[mine].max((0, 2))
                    s = got[2 + which][blk].astype(np.float64)
                    old = (self.ks, self.vs)[which][blk].astype(np.float64) if c > b * u else np.zeros(nkv)
                    low, high = np.maximum(old, scale_of(amax - edge)), np.maximum(old, scale_of(amax + edge))
                    assert np.all((s == low) | (s == high)), f"sequence {i} block {b}: scale {s} for {amax}"
                    sb = s[None, :, None]
                    y = E4M3[got[which][slots[mine]]] * sb
                    assert np.all(np.abs(y - want[mine]) <= tol[mine] + np.maximum(2.0 ** -4 * np.abs(want[mine]), 2.0 ** -10 * sb)
                                  + 1e-300), f"sequence {i} block {b}: pool {which}"
                    if which == 1 and np.all(s > 0):  # V is not computed: its codes are exact
                        assert np.array_equal(got[1][slots[mine]], to_e4m3((want[mine].astype(np.float32) / sb.astype(np.float32))))
                    before = np.arange(b * u, max(c, b * u))
                    if c > b * u and len(before):
                        ps = self.slots(i, before)
                        touched[ps] = True
                        was = (self.k, self.v)[which][ps]
                        grown = s > old
                        then = to_e4m3((E4M3[was].astype(np.float32) * old[None, :, None].astype(np.float32))
                                       / sb.astype(np.float32))
                        assert np.array_equal(got[which][ps], np.where(grown[None, :, None], then, was)), "requantised"
                    pools[2 + which][blk] = got[2 + which][blk]
        for which in (0, 1):
            assert np.array_equal(got[which][~touched], pools[which][~touched]), "wrote past the new tokens"
            if self.bits == 8:
                assert np.array_equal(got[2 + which], pools[2 + which]), "another block's scale"
        return owned


SHAPES = [(16, 2, 256, 16, 16), (8, 1, 128, 32, 16), (32, 8, 128, 64, 64), (24, 2, 256, 128, 128), (6, 2, 128, 96, 32),
          (4, 4, 256, 64, 16)]


@pytest.mark.parametrize("nq,nkv,hd,page,unit", SHAPES)
def test_ragged_8(qsa, nq, nkv, hd, page, unit):
    """Blocks begun and fresh, one token and many, sequences without rows, rows of no sequence."""
    rng = qi.rng_for(50, salt=nq + hd + unit)
    c = Write(qsa, rng, [0, 1, unit - 1, unit, unit + 1, 5 * unit + 3, 40, 2 * unit], [1, 2 * unit, 1, 1, unit - 1, 3 * unit + 1, 0, unit],
              nq, nkv, hd, page, unit, gaps=2)
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    owned = c.check(o, got)
    assert np.all(o[~owned] == SENT) and (~owned).sum() == 4
    again, got2, _ = c.run(qsa, inplace=True)
    assert np.array_equal(again[owned], o[owned]) and np.array_equal(again[~owned], c.x[~owned, :nq * hd])
    assert all(np.array_equal(a, b) for a, b in zip(got, got2))


@pytest.mark.parametrize("nq,nkv,hd,page", [(16, 2, 256, 16), (8, 1, 128, 7), (6, 2, 128, 100), (12, 4, 256, 1)])
def test_ragged_bf16(qsa, nq, nkv, hd, page):
    rng = qi.rng_for(51, salt=nq + hd + page)
    c = Write(qsa, rng, [0, 1, 15, 16, 17, 83, 40], [1, 33, 1, 1, 15, 49, 0], nq, nkv, hd, page, bits=16, gaps=1)
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    owned = c.check(o, got)
    assert np.all(o[~owned] == SENT)


@pytest.mark.parametrize("n,rows", [(1, 1), (70, 1), (3, 700), (600, 2)])
@pytest.mark.parametrize("bits", [8, 16])
def test_steps_and_chunks(qsa, n, rows, bits):
    """More sequences than a warp's lanes and a CTA's threads, a long chunk; positions of their own."""
    rng = qi.rng_for(52, salt=n + bits)
    ctx = rng.integers(0, 90, n)
    c = Write(qsa, rng, ctx, [rows] * n, 8, 2, 128, 32, 32, bits, pos=rng.integers(0, 900, n * rows).astype(np.int32), table_rows=900)
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    c.check(o, got)


def test_no_norm(qsa):
    rng = qi.rng_for(53)
    c = Write(qsa, rng, [7], [40], 4, 2, 128, 16, 16, norm=False)
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    c.check(o, got)


def test_scales_at_their_edges(qsa):
    """V heads whose largest value is 448 * 2^k or next to it, zero blocks, tiny and huge values, a scale that stays."""
    rng = qi.rng_for(54)
    tops = np.array([448.0, 450.0, 446.0, 224.0, 1.75 * 2.0 ** -60, 2.0 ** 120, 0.0, 7.0], np.float32)
    c = Write(qsa, rng, [5] * 8, [16] * 8, 2, 1, 128, 32, 16)
    x = c.x.copy()
    for i, top in enumerate(tops):
        v = f64(x[16 * i:16 * i + 16, 384:512])
        x[16 * i:16 * i + 16, 384:512] = qi.to_bf16_bits((v / np.abs(v).max() * 0.9 * top).astype(np.float32))
        for r in (3, 13):  # one in the begun block, one in the fresh one
            x[16 * i + r, 384 + r] = qi.to_bf16_bits(np.array([-top], np.float32))[0]
    c.x = x
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    c.check(o, got)
    fresh = np.array([c.slots(i, 16) // 16 for i in range(8)])
    assert np.array_equal(got[3][fresh, 0], scale_of(f64(qi.to_bf16_bits(tops))).astype(np.float32))
    assert np.all(got[1][c.slots(6, np.arange(16, 21))] & 0x7F == 0) and got[3][fresh[6], 0] == 0


def test_a_zero_block_grows(qsa):
    """A begun block of scale 0 takes the new one's scale; its tokens stay zero."""
    rng = qi.rng_for(55)
    c = Write(qsa, rng, [9], [3], 2, 1, 128, 16, 16)
    blk = int(c.slots(0, 0)) // 16
    c.vs[blk] = 0
    c.v[c.slots(0, np.arange(9))] = 0
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    c.check(o, got)
    assert got[3][blk, 0] > 0 and np.all(got[1][c.slots(0, np.arange(9))] == 0)


def test_a_scale_that_grows_by_steps(qsa):
    """One token at a time into a block, each larger: the block's values stay what they were, up to its rounding."""
    rng = qi.rng_for(56)
    c = Write(qsa, rng, [0], [1], 2, 1, 128, 16, 16, table_rows=16)
    c.pos = np.array([3], np.int32)
    first = None
    for t in range(16):
        c.ctx, c.x = np.array([t], np.int32), qi.normal_bf16(rng, c.x.shape, std=2.0 ** (t / 2 - 3))
        o, got, st = c.run(qsa)
        assert st == (0, 0)
        c.check(o, got)
        c.k, c.v, c.ks, c.vs = got
        if t == 0:
            first = f64(c.x[0, 384:512])
    s = float(c.vs[int(c.slots(0, 0)) // 16, 0])
    held = E4M3[c.v[c.slots(0, 0)][0]] * s
    # each growth of the scale may round once more below 2^-6 s: 2^-10 of that scale, and scales double at least
    assert np.all(np.abs(held - first) <= 2.0 ** -4 * np.abs(first) + 2 * 2.0 ** -10 * s)


@pytest.mark.parametrize("bits", [8, 16])
def test_values_that_are_not_finite(qsa, bits):
    """A NaN or an infinity of V is held as NaN (bf16: as it is); the block's other values and its scale do not see it."""
    rng = qi.rng_for(57)
    c = Write(qsa, rng, [4], [20], 2, 1, 128, 16, 16, bits)
    o, clean, _ = c.run(qsa)
    for word in qi.to_bf16_bits(np.array([np.nan, np.inf, -np.inf], np.float32)):
        x = c.x.copy()
        c.x[7, 384 + 5] = word
        c.x[7, 384 + 6] = 0
        _, got, st = c.run(qsa)
        assert st == (0, 0)
        slot = c.slots(0, 11)
        if bits == 8:
            assert got[1][slot, 0, 5] & 0x7F == 0x7F
            same = got[1] == clean[1]
            same[slot, 0, 5:7] = True
            assert np.all(same) and np.array_equal(got[3], clean[3]) and np.array_equal(got[0], clean[0])
        else:
            assert got[1][slot, 0, 5] == word
        c.x = x


@pytest.mark.parametrize("bits", [8, 16])
def test_positions_out_of_range(qsa, bits):
    rng = qi.rng_for(58)
    for bad in (-1, 50, 2 ** 31 - 1, -2 ** 31):
        pos = np.arange(30, dtype=np.int32)
        pos[[3, 12, 29]] = bad
        c = Write(qsa, rng, [5, 0], [13, 17], 4, 2, 128, 16, 16, bits, pos=pos, table_rows=50)
        o, got, st = c.run(qsa)
        assert st in ((3, 0), (3, 1))
        owned = c.check(o, got, left_alone=(3, 12, 29))
        assert np.all(o[[3, 12, 29]] == SENT) and owned.sum() == 27
    # a block none of whose rows is good stays as it is
    pos[:] = bad
    c = Write(qsa, rng, [5], [30], 4, 2, 128, 16, 16, bits, pos=pos, table_rows=50)
    o, got, st = c.run(qsa)
    assert st == (3, 0) and np.all(o == SENT)
    assert all(np.array_equal(a, b) for a, b in zip(got, (c.k, c.v, c.ks, c.vs)) if b is not None)


@pytest.mark.parametrize("bits", [8, 16])
def test_bad_sequences_and_pages(qsa, bits):
    rng = qi.rng_for(59)
    for which in range(4):
        c = Write(qsa, rng, [20, 7, 33], [5, 30, 9], 4, 2, 128, 16, 16, bits)
        good = [0, 2]
        if which == 0:
            c.ctx[1] = -1
        elif which == 1:
            c.ctx[1] = c.table_len * 16 - 29
        elif which == 2:
            c.ctx[1] = 2 ** 31 - 5
        else:
            c.table[1, 1] = c.pages + (0 if bits == 8 else 100)
        cos_rows = 64
        c.table_rows = cos_rows
        c.cos, c.sin = qsa.qsa_rope_tables(cos_rows, 10000.0)
        o, got, st = c.run(qsa)
        assert st == ((3, 1) if which < 3 else (6, 1))
        if which < 3:
            assert np.all(o[5:35] == SENT)
            c.rows, c.n = np.array([5, 0, 9], np.int32), 3
            c.ctx[1] = 0
            c.check(o, got)
        else:  # its queries are done, its tokens of the other pages too
            assert np.all(o != SENT)
            inside = c.slots(1, np.arange(7, 16))
            if bits == 16:
                assert not np.array_equal(got[0][inside], c.k[inside])


def test_starts_that_do_not_ascend(qsa):
    """A bad sequence is left out alone, also where its start lies above those behind it."""
    rng = qi.rng_for(60)
    for n in (4, 40):
        c = Write(qsa, rng, [20] * n, [5] * n, 4, 2, 128, 32, 16)
        o, clean, _ = c.run(qsa)
        c.row_start[1] = c.n_rows + 50
        o2, got, st = c.run(qsa)
        assert st[0] == 3 and st[1] in (0, 1)
        assert np.all(o2[:10] == SENT) and np.array_equal(o2[10:], o[10:])


def test_streams_and_graphs(qsa):
    rng = qi.rng_for(61)
    c = Write(qsa, rng, [5, 30], [40, 3], 8, 2, 128, 16, 16)
    o, got, _ = c.run(qsa)
    o2, got2, _ = c.run(qsa, stream=torch.cuda.Stream())
    assert np.array_equal(o, o2) and all(np.array_equal(a, b) for a, b in zip(got, got2))
