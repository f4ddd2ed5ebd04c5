"""Cases and plain forms in 64 bits shared by the tests of the step operators (page
plans, the write of prepared heads into the cache, attention over an 8-bit cache).

Tolerances, from the arithmetic (U = 2^-24, a rounding to f32; 2^-8 one to bf16, 2^-4
one to e4m3, whose steps below 2^-6 are 2^-9 each).

Write: a head's sum of squares runs in f32 over 8 terms a lane and 5 sums of lanes, the
reciprocal root is off by 2^-22.9, x r (1 + w) rounds three times: under 16 U of a value
together, and a turned value x c + y s adds 2 U (|x c| + |y s|).

Attention: a logit is scale ks sum q_d k_d, accumulated in f32 whose adder may
truncate: off by at most delta = |scale| ks ((hd + 8) 2 U sum |q_d k_d| +
2^-17 max |q| sum |k_d|), the second for what is left of q's two e4m3 terms.  A weight
times its V scale is held as two e4m3 terms: off by 2^-8 of itself or by 2^-18 of the
row's largest one.
"""
import numpy as np
import torch

import qsa_inputs as qi
from cache_cases import BF, U, dev, f64

_codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
E4M3 = _codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()  # value of each code; NaN for 0x7F and 0xFF


def to_e4m3(x):
    """Codes of the nearest e4m3 values (|x| <= 448), ties to even: from the table of values."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy().copy()


def scale_of(amax):
    """The least power of two s with amax <= 448 s."""
    m, e = np.frexp(np.asarray(amax, np.float64))
    return np.where(amax > 0, np.ldexp(1.0, e - 9 + (m > 0.875)), 0.0)


def pool_8(rng, tokens, nkv, hd, unit, std=1.0, spread=0.5):
    """Codes [tokens, nkv, hd] and scales [tokens / unit, nkv] (no powers of two) of a random pool."""
    x = rng.standard_normal((tokens // unit, unit, nkv, hd)) * std * np.exp(spread * rng.standard_normal((tokens // unit, 1, nkv, 1)))
    s = (np.abs(x).max((1, 3)) / rng.uniform(200, 448)).astype(np.float32)
    return to_e4m3((x / s[:, None, :, None]).reshape(tokens, nkv, hd)), s


class Cache8:
    """n sequences' paged 8-bit K/V (shuffled pages) and their drafted rows."""

    def __init__(self, rng, ctx, rows, nq, nkv, hd, page, unit, mask="tree", gaps=0, q_std=1.5, n_first=0, window=0, words=None):
        self.ctx, self.rows = np.asarray(ctx, np.int32), np.asarray(rows, np.int32)
        self.nq, self.nkv, self.hd, self.page, self.unit = nq, nkv, hd, page, unit
        self.n_first, self.window = n_first, window
        self.n, self.group = len(ctx), nq // nkv
        per = np.maximum(1, -(-(self.ctx + self.rows) // page))
        self.table_len, self.pages = int(per.max()), int(per.sum()) + 2
        order = rng.permutation(self.pages)
        self.table = np.full((self.n, self.table_len), -1, np.int32)
        at = 0
        for i, p in enumerate(per):
            self.table[i, :p] = order[at:at + p]
            at += int(p)
        self.k, self.ks = pool_8(rng, self.pages * page, nkv, hd, unit, spread=0.2)
        self.v, self.vs = pool_8(rng, self.pages * page, nkv, hd, unit)
        self.row_start = (np.concatenate([[0], np.cumsum(self.rows)]) + gaps).astype(np.int32)
        self.n_rows = int(self.row_start[-1]) + gaps
        self.q = qi.normal_bf16(rng, (self.n_rows, nq * hd), std=q_std)
        self.mask, self.words = None, 0
        if mask != "chain":
            most = max(1, int(self.rows.max()))
            self.words = (most + 31) // 32 if words is None else words
            self.mask = rng.integers(0, 1 << 32, size=(self.n_rows, self.words), dtype=np.uint32)
            if mask == "tree":  # ancestors and itself; bits past the drafted tokens stay random
                for i in range(self.n):
                    m = int(self.rows[i])
                    sees = np.zeros((m, m), bool)
                    for j in range(m):
                        p = int(rng.integers(max(-1, j - 4), j)) if j else -1
                        if p >= 0:
                            sees[j] = sees[p]
                        sees[j, j] = True
                    self.set_bits(i, sees)

    def set_bits(self, i, sees):
        r0, m = int(self.row_start[i]), int(self.rows[i])
        bits = np.unpackbits(self.mask[r0:r0 + m].view(np.uint8), axis=1, bitorder="little")
        bits[:, :m] = sees
        self.mask[r0:r0 + m] = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)

    def slots(self, i, tokens):
        tokens = np.asarray(tokens)
        return self.table[i, tokens // self.page].astype(np.int64) * self.page + tokens % self.page

    def sees(self, i):
        """[m, kv]: which cached tokens each row of sequence i sees."""
        m, c = int(self.rows[i]), int(self.ctx[i])
        r0, j, t = int(self.row_start[i]), np.arange(m)[:, None], np.arange(c + m)[None]
        near = np.ones((m, c + m), bool)
        if self.mask is None:
            if self.window:
                near = (t < self.n_first) | (c + j - t < self.window)
            return near & (t <= c + j)
        bits = np.unpackbits(self.mask[r0:r0 + m].view(np.uint8), axis=1, bitorder="little")[:, :m].astype(bool)
        if self.window:
            p = c + np.maximum(0, bits.sum(1, keepdims=True) - 1)
            near = (t < self.n_first) | (p - t < self.window)
        return np.concatenate([near[:, :c], bits], 1)

    def kv(self, i):
        """The sequence's K and V in 64 bits and their codes' values and scales: each [kv, nkv, ...]."""
        at = self.slots(i, np.arange(int(self.ctx[i] + self.rows[i])))
        k8, v8 = E4M3[self.k[at]], E4M3[self.v[at]]
        ks, vs = self.ks[at // self.unit].astype(np.float64), self.vs[at // self.unit].astype(np.float64)
        return k8 * ks[:, :, None], v8 * vs[:, :, None], v8, vs

    def args(self, q_d, q_stride, d=None):
        d = self.device() if d is None else d
        return (q_d, q_stride, self.nq, self.nkv, self.hd, d["k"], d["v"], d["ks"], d["vs"], self.unit, self.pages, self.page,
                d["table"], self.table_len, self.table_len, d["ctx"], d["start"], self.n, self.n_rows, d["mask"], self.words,
                self.n_first, self.window)

    def device(self):
        return dict(k=dev(self.k), v=dev(self.v), ks=dev(self.ks), vs=dev(self.vs), table=dev(self.table), ctx=dev(self.ctx),
                    start=dev(self.row_start), mask=None if self.mask is None else dev(self.mask))


def ref_attend(c, i, scale):
    """Output [m, nq, hd], lse [m, nq] and their bounds, in 64 bits."""
    m, r0 = int(c.rows[i]), int(c.row_start[i])
    q = f64(c.q[r0:r0 + m]).reshape(m, c.nq, c.hd)
    k, v, v8, vs = c.kv(i)
    vis = c.sees(i)
    out, tol = np.zeros((m, c.nq, c.hd)), np.zeros((m, c.nq, c.hd))
    lse, ltol = np.full((m, c.nq), -np.inf), np.zeros((m, c.nq))
    for j in range(m):
        t = np.nonzero(vis[j])[0]
        if len(t) == 0:
            continue
        for g in range(c.nkv):
            heads = slice(g * c.group, (g + 1) * c.group)
            qg, n = q[j, heads], len(t)
            with np.errstate(all="ignore"):
                s = (qg @ k[t, g].T) * scale
                ak = np.abs(k[t, g])
                delta = abs(scale) * np.max((c.hd + 8) * 2 * U * (np.abs(qg) @ ak.T)
                                            + 2.0 ** -17 * np.abs(qg).max(1, keepdims=True) * ak.sum(1)[None], axis=1)
                top = s.max(1)
                p = np.exp(s - top[:, None])
                lse[j, heads] = top + np.log(p.sum(1))
                p /= p.sum(1, keepdims=True)
                out[j, heads] = p @ v[t, g]
                weight = p @ np.abs(v[t, g])
                floor = 2.0 ** -18 * (p * vs[t, g][None]).max(1)[:, None] * np.abs(v8[t, g]).sum(0)[None]
            tol[j, heads] = (BF + 4 * delta[:, None] + 2.0 ** -20 + 2 * n * U) * weight + floor + BF * np.abs(out[j, heads]) + 1e-30
            ltol[j, heads] = delta + n * U + 2.0 ** -20 + 4 * U * np.abs(lse[j, heads])
    return out, tol, lse, ltol


def ref_plan(ctx, new, page, table, held, free, n_free, max_rows, pool_pages):
    """The outputs of a page plan and its status code and row, one step after another."""
    n, table_len = table.shape
    table, free, held = table.copy(), free.copy(), held.copy()
    out = dict(table=table, free=free, held=held, n_free=n_free, row_start=np.zeros(n + 1, np.int32),
               slot=np.full(max_rows, -1, np.int32), pos=np.zeros(max_rows, np.int32), row_seq=np.full(max_rows, -1, np.int32))
    ok = [ctx[s] >= 0 and new[s] >= 0 and 0 <= held[s] <= table_len and int(ctx[s]) + int(new[s]) <= table_len * page
          for s in range(n)]
    errors = [(3, s) for s in range(n) if not ok[s]]
    rows = [int(new[s]) if ok[s] else 0 for s in range(n)]
    need = [-(-(int(ctx[s]) + rows[s]) // page) if ok[s] else int(held[s]) for s in range(n)]
    back = sum(max(0, int(held[s]) - need[s]) for s in range(n))
    take = np.cumsum([max(0, need[s] - int(held[s])) for s in range(n)])
    if n_free < 0 or n_free + back > pool_pages:
        return out, errors + [(6, 0)]
    if sum(rows) > max_rows:
        return out, errors + [(3, int(np.nonzero(np.cumsum(rows) > max_rows)[0][0]))]
    if take[-1] > n_free + back:
        return out, errors + [(7, int(np.nonzero(take > n_free + back)[0][0]))]
    for s in range(n):
        for e in range(need[s], int(held[s])):
            free[n_free] = table[s, e]
            n_free += 1
    for s in range(n):
        for e in range(int(held[s]), need[s]):
            n_free -= 1
            table[s, e] = free[n_free]
    r = 0
    for s in range(n):
        out["row_start"][s] = r
        for j in range(rows[s]):
            t = int(ctx[s]) + j
            out["slot"][r], out["pos"][r], out["row_seq"][r] = table[s, t // page] * page + t % page, t, s
            r += 1
        held[s] = need[s]
    out["row_start"][n] = r
    out["n_free"] = n_free
    return out, errors


def ref_heads(x, w, eps, cos, sin):
    """Heads x [rows, heads, hd] normed (w None: not) and turned by cos, sin [rows, 64], and the bound of f32."""
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 + w)
    out, mag = y.copy(), np.abs(y)
    if cos is not None:
        c, s = cos[:, None, :32], sin[:, None, :32]
        a, b = y[..., :32], y[..., 32:64]
        out[..., :32], out[..., 32:64] = a * c - b * s, b * c + a * s
        mag[..., :32], mag[..., 32:64] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, 18 * U * mag
