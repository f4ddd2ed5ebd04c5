"""Cases and 64-bit plain forms shared by the tests of the cache operators
(tree attention, attention mass, eviction, compaction).

Tolerances, from the arithmetic (u = 2^-24, a rounding to f32; 2^-8, one to
bf16).  A logit is a sum of head_dim exact products accumulated in f32, whose
adder may truncate (2u a step): off by at most
    delta = scale * (head_dim + 4) * 2u * sum_d |q_d k_d|
with the scale's own rounding and the exponent's in the 4.  A weight exp(s - lse)
is then off by at most 2 delta + 2^-21 of itself (ex2's error is under 2^-22,
|s - max| log2(e) in one rounding adds |s - max| u, covered by the sum in
delta), its rounding to bf16 by 2^-8, and an f32 sum of n terms by n u.
"""
import numpy as np
import torch

import qsa_inputs as qi

U = 2.0 ** -24
BF = 2.0 ** -8


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    return torch.from_numpy(a).cuda()


def f64(bits):
    return qi.bf16_bits_to_f32(bits).astype(np.float64)


class Cache:
    """n sequences' paged K/V (shuffled pages) and their drafted rows."""

    def __init__(self, rng, ctx, rows, nq, nkv, hd, page, mask="tree", words=None, gaps=0, q_std=1.5):
        self.ctx, self.rows = np.asarray(ctx, np.int32), np.asarray(rows, np.int32)
        self.nq, self.nkv, self.hd, self.page = nq, nkv, hd, page
        self.n, self.group = len(ctx), nq // nkv
        kv = self.ctx + self.rows
        per = np.maximum(1, -(-kv // page))
        self.table_len = int(per.max())
        self.pages = int(per.sum()) + 2
        order = rng.permutation(self.pages)
        self.table = np.full((self.n, self.table_len), -1, np.int32)
        at = 0
        for i, p in enumerate(per):
            self.table[i, :p] = order[at:at + p]
            at += int(p)
        width = nkv * hd
        self.k = qi.normal_bf16(rng, (self.pages * page, width))
        self.v = qi.normal_bf16(rng, (self.pages * page, width))
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
        for j in range(m):
            for k in range(m):
                w, b = k // 32, np.uint32(1 << (k % 32))
                self.mask[r0 + j, w] = (self.mask[r0 + j, w] | b) if sees[j, k] else (self.mask[r0 + j, w] & ~b)

    def sees(self, i):
        m = int(self.rows[i])
        if self.mask is None:
            return np.tril(np.ones((m, m), bool))
        r0 = int(self.row_start[i])
        bits = np.unpackbits(self.mask[r0:r0 + m].view(np.uint8), axis=1, bitorder="little")
        return bits[:, :m].astype(bool)

    def slots(self, i, tokens):
        tokens = np.asarray(tokens)
        return self.table[i, tokens // self.page].astype(np.int64) * self.page + tokens % self.page

    def seq(self, i):
        """q [m, nq, hd], K, V [kv, nkv, hd] in 64 bits, visibility [m, kv]."""
        m, c = int(self.rows[i]), int(self.ctx[i])
        r0 = int(self.row_start[i])
        at = self.slots(i, np.arange(c + m))
        vis = np.concatenate([np.ones((m, c), bool), self.sees(i)], axis=1)
        return (f64(self.q[r0:r0 + m]).reshape(m, self.nq, self.hd),
                f64(self.k[at]).reshape(-1, self.nkv, self.hd), f64(self.v[at]).reshape(-1, self.nkv, self.hd), vis)

    def tree_args(self, q_d, q_stride, dk=None, dv=None):
        d = self.device()
        return (q_d, q_stride, self.nq, self.nkv, self.hd, d["k"], d["v"], self.pages, self.page, d["table"],
                self.table_len, self.table_len, d["ctx"], d["start"], self.n, self.n_rows, d["mask"], self.words)

    def mass_args(self, q_d, q_stride):
        a = self.tree_args(q_d, q_stride)
        return a[:6] + a[7:]

    def device(self):
        return dict(k=dev(self.k), v=dev(self.v), table=dev(self.table), ctx=dev(self.ctx), start=dev(self.row_start),
                    mask=None if self.mask is None else dev(self.mask))


def ref_tree(c, i, scale):
    """Output [m, nq, hd], lse [m, nq] and their bounds, in 64 bits."""
    q, k, v, vis = c.seq(i)
    m = q.shape[0]
    out, tol = np.zeros((m, c.nq, c.hd)), np.zeros((m, c.nq, c.hd))
    lse, ltol = np.full((m, c.nq), -np.inf), np.zeros((m, c.nq))
    for j in range(m):
        t = np.nonzero(vis[j])[0]
        if len(t) == 0:
            continue
        for h in range(c.nq):
            g = h // c.group
            with np.errstate(all="ignore"):
                s = (k[t, g] @ q[j, h]) * scale
                delta = abs(scale) * (c.hd + 4) * 2 * U * float((np.abs(k[t, g]) @ np.abs(q[j, h])).max())
                top = s.max()
                p = np.exp(s - top)
                lse[j, h] = top + np.log(p.sum())
                p = p / p.sum()
                out[j, h] = p @ v[t, g]
                weight = p @ np.abs(v[t, g])
            n = len(t)
            tol[j, h] = (BF + 4 * delta + 2 ** -20 + 2 * n * U) * weight + BF * np.abs(out[j, h]) + 1e-30
            ltol[j, h] = delta + n * U + 2 ** -20 + 4 * U * abs(lse[j, h])
    return out, tol, lse, ltol


def ref_mass(c, i, scale, lse, weight, carry, old):
    """Mass [nkv, kv] of sequence i and its bound; lse [m, nq] f32, old [nkv, >= kv]."""
    q, k, _, vis = c.seq(i)
    m, kv, ctx = q.shape[0], k.shape[0], int(c.ctx[i])
    r0 = int(c.row_start[i])
    got = np.zeros((c.nkv, kv))
    got[:, :ctx] = old[:, :ctx].astype(np.float64) * carry if carry else 0.0
    tol = 3 * U * np.abs(got)
    for g in range(c.nkv):
        for j in range(m):
            w = 1.0 if weight is None else float(weight[r0 + j])
            if w == 0:
                continue
            for h in range(g * c.group, (g + 1) * c.group):
                if lse[j, h] == -np.inf:
                    continue
                t = vis[j]
                s = (k[t, g] @ q[j, h]) * scale
                delta = abs(scale) * (c.hd + 4) * 2 * U * (np.abs(k[t, g]) @ np.abs(q[j, h]))
                p = w * np.exp(s - float(lse[j, h]))
                got[g, t] += p
                tol[g, t] += np.abs(p) * (2 * delta + 2 ** -20 + 4 * U * abs(float(lse[j, h])) + 2 * m * c.group * U)
    return got, tol + 1e-30


def keep_units(mass, length, keep, first, last, unit):
    """The kept tokens of one sequence; mass [nkv, cols] f32, sums in the documented f32 order."""
    units = length // unit
    if units <= keep // unit:
        return np.arange(length)
    tok = mass[0, :length].copy()
    for h in range(1, mass.shape[0]):
        tok = (tok + mass[h, :length]).astype(np.float32)
    u = tok[:units * unit].reshape(units, unit)
    score = u[:, 0].copy()
    for e in range(1, unit):
        score = (score + u[:, e]).astype(np.float32)
    always = np.zeros(units, bool)
    always[:first // unit] = True
    always[units - last // unit:] = True
    order = sorted(range(units), key=lambda x: (not always[x], -float(score[x]) + 0.0, x))
    stay = np.sort(np.array(order[:keep // unit], np.int64))
    return np.concatenate([(stay[:, None] * unit + np.arange(unit)).reshape(-1), np.arange(units * unit, length)])
