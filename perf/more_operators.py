"""Cases of the step operators: the pages, rows and slots of a step, the norm and rotation of its
queries and keys on their way into the cache, and attention over a cache held in 8 bits.

With ``own`` false ``run`` computes each operator from elementary torch operations in 32 bits (the
norms and rotated keys in 64: their 8-bit values round at borders); with ``own`` true it calls the
library.  ``exact`` computes the same results in 64 bits, one sequence at a time.  Lengths and row
counts follow from a case alone, contents from the seed.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
EIGHT = torch.float8_e4m3fn
MOST_8 = 448.0  # the largest e4m3 value


def listed():
    return [
        # --- pages, rows and slots of a step
        # a decode step of a serving batch: one token each, some at the end of a page
        dict(name="plan decode 64", op="plan", n=64, lo=300, hi=9001, rlo=1, rhi=1, page=16, slack=0, shape=21),
        # many requests at once, prompts among them; some shrank since the last step and give pages back
        dict(name="plan 1024 ragged", op="plan", n=1024, lo=0, hi=32768, rlo=0, rhi=257, page=16, slack=40, shape=22),
        # --- norms and rotation of queries and keys, the cache write
        # one sequence early in its answer: latency is all
        dict(name="write one row 515", op="write", n=1, lo=515, hi=515, rlo=1, rhi=1, nq=16, nkv=2, hd=256, page=16, unit=16,
             held=8, shape=23),
        # a decode batch: one token each into blocks that are partly full
        dict(name="write decode 64", op="write", n=64, lo=300, hi=4099, rlo=1, rhi=1, nq=32, nkv=8, hd=128, page=64, unit=64,
             held=8, shape=24),
        # a chunk of a long prompt
        dict(name="write chunk 4096", op="write", n=1, lo=4100, hi=4100, rlo=4096, rhi=4096, nq=16, nkv=2, hd=256, page=16,
             unit=16, held=8, shape=25),
        # several prompts of odd lengths, the cache in bf16
        dict(name="write bf16 8 prompts", op="write", n=8, lo=0, hi=33, rlo=101, rhi=777, nq=32, nkv=8, hd=128, page=64, unit=64,
             held=16, shape=26),
        # --- attention over a cache held in 8 bits
        # one sequence early in its answer, one token at a time
        dict(name="attend one row 515", op="attend", n=1, lo=515, hi=515, rlo=1, rhi=1, nq=16, nkv=2, hd=256, page=16, unit=16,
             mask="chain", first=0, window=0, shape=27),
        # a decode batch: every sequence's whole cache read for one row
        dict(name="attend decode 16x64k", op="attend", n=16, lo=16384, hi=65535, rlo=1, rhi=1, nq=16, nkv=2, hd=256, page=16,
             unit=16, mask="chain", first=0, window=0, shape=28),
        # one long sequence verifying a tree of 64 drafted tokens
        dict(name="attend verify 64 of 64k", op="attend", n=1, lo=65471, hi=65471, rlo=64, rhi=64, nq=16, nkv=2, hd=256, page=16,
             unit=16, mask="tree", first=0, window=0, shape=29),
        # a serving batch verifying small trees of odd sizes over short and middle contexts
        dict(name="attend verify batch", op="attend", n=24, lo=300, hi=9001, rlo=5, rhi=37, nq=32, nkv=8, hd=128, page=64, unit=64,
             mask="tree", first=0, window=0, shape=30),
        # long sequences of a layer that looks back 4096 tokens and at the first 16
        dict(name="attend window 4096 of 64k", op="attend", n=16, lo=16384, hi=65535, rlo=1, rhi=1, nq=16, nkv=2, hd=256, page=16,
             unit=16, mask="chain", first=16, window=4096, shape=31),
        # a chunk of a prompt in a layer of the same kind, a shorter window
        dict(name="attend window chunk 2048", op="attend", n=1, lo=6001, hi=6001, rlo=2048, rhi=2048, nq=32, nkv=8, hd=128, page=64,
             unit=64, mask="chain", first=4, window=1024, shape=32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "write", "attend", "attend", "attend", "attend"])
    if op == "plan":
        n = _log_int(rng, 1, 1024)
        hi, rhi = _log_int(rng, 1, 32768), _log_int(rng, 1, 400)
        return dict(op=op, n=n, lo=rng.randint(0, hi), hi=hi, rlo=rng.randint(0, rhi), rhi=rhi,
                    page=rng.choice([1, 7, 16, 32, 64, 100, 256]), slack=rng.choice([0, 0, 5, 60]), shape=rng.randrange(1 << 30))
    nq, nkv, hd = rng.choice([(16, 2, 256), (32, 8, 128), (8, 1, 128), (24, 2, 256), (6, 2, 128), (12, 4, 256), (4, 4, 128)])
    n = _log_int(rng, 1, 40)
    unit = rng.choice([16, 16, 32, 64, 128])
    c = dict(op=op, n=n, nq=nq, nkv=nkv, hd=hd, unit=unit, page=unit * rng.choice([1, 1, 2, 3]), shape=rng.randrange(1 << 30))
    if op == "write":
        hi, rhi = _log_int(rng, 1, 4099), _log_int(rng, 1, max(2, 8192 * 1024 // (n * nq * hd // 2)))
        return dict(c, lo=rng.randint(0, hi), hi=hi, rlo=rng.randint(0, rhi), rhi=rhi, held=rng.choice([8, 8, 16]))
    width = nkv * hd
    hi = _log_int(rng, 1, max(2, min(65536, 1000000000 // (n * width * 4))))
    c.update(lo=max(0, hi // rng.randint(1, 8) - 1), hi=hi)
    rows_most = max(1, min(160, int(5e10 / (4.0 * n * nq * hd * (hi + 128)))))
    rhi = _log_int(rng, 1, rows_most)
    c.update(rlo=rng.randint(1, rhi), rhi=rhi, mask=rng.choice(["tree", "chain"]), first=0, window=0)
    if rng.random() < 0.4:
        c.update(first=rng.choice([0, 1, 4, 16, 130]), window=_log_int(rng, 1, 8192))
    return c


# ---------------------------------------------------------------- shapes and inputs

def _shapes(case):
    """Cached lengths and row counts of a case: numpy int arrays."""
    r = np.random.RandomState(case["shape"] % (1 << 31))
    ctx = r.randint(case["lo"], case["hi"] + 1, size=case["n"]).astype(np.int64)
    rows = r.randint(case["rlo"], case["rhi"] + 1, size=case["n"]).astype(np.int64)
    if case["op"] == "write" and not rows.any():
        rows[0] = 1
    return ctx, rows


def _held(case):
    """Pages that each sequence of a plan holds: those of its context, and up to `slack` more."""
    ctx, _ = _shapes(case)
    r = np.random.RandomState((case["shape"] + 1) % (1 << 31))
    return -(-ctx // case["page"]) + r.randint(0, case["slack"] + 1, size=case["n"]) * (r.rand(case["n"]) < 0.25)


def work(case):
    ctx, rows = _shapes(case)
    total = int(rows.sum())
    if case["op"] == "plan":
        n, page = case["n"], case["page"]
        moved = int(np.abs(-(-(ctx + rows) // page) - _held(case)).sum())
        return dict(bytes=4 * (3 * n + 1) + 4 * (2 * n + 2) + 8 * moved + 12 * total, flops=4 * total + 8 * n)
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    if case["op"] == "write":
        b = 2 * total * (nq + 2 * nkv) * hd + 2 * total * nq * hd + total * 256 + 2 * total * nkv * hd * (case["held"] // 8)
        if case["held"] == 8:
            blocks = int(((ctx + rows + case["unit"] - 1) // case["unit"] - ctx // case["unit"])[rows > 0].sum())
            b += 8 * nkv * blocks
        return dict(bytes=b, flops=total * ((nq + nkv) * (4 * hd + 3 * 64) + 4 * nkv * hd))
    pairs = seen = 0
    for c, m in zip(ctx.tolist(), rows.tolist()):
        if not case["window"]:
            pairs, seen = pairs + m * c + m * (m + 1) // 2, seen + c + m
            continue
        first, w = min(case["first"], c), case["window"]
        p = c + np.arange(m)
        lo = np.maximum(first, p - w + 1)
        pairs, seen = pairs + int((first + np.maximum(0, p + 1 - lo)).sum()), seen + first + max(0, c + m - int(lo[0]))
    b = 2 * seen * nkv * hd + 8 * nkv * (seen // case["unit"]) + 4 * total * nq * hd + 4 * total * nq
    return dict(bytes=b, flops=4 * pairs * nq * hd)


def _tree_bits(r, rows, words):
    """Which drafted tokens each drafted row sees, itself among them: uint32 words [sum(rows), words]."""
    n, most = len(rows), int(rows.max())
    sees = np.zeros((n, most, most), bool)
    for k in range(most):  # a token's parent is an earlier one, or the context (-1)
        if k:
            parent = np.maximum(-1, k - r.geometric(0.4, size=n))
            has = parent >= 0
            sees[has, k] = sees[np.nonzero(has)[0], parent[has]]
        sees[:, k, k] = True
    flat = np.concatenate([sees[i, :rows[i]] for i in range(n)])
    bits = np.zeros((flat.shape[0], words * 32), np.uint8)
    bits[:, :most] = flat
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEVICE)


def _normal(gen, shape, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * std).to(torch.bfloat16)


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8); 0 for amax 0."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1
    e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _over(x, scale):
    return torch.where(scale > 0, x / torch.where(scale > 0, scale, torch.ones_like(scale)), torch.zeros_like(x))


def _pool_8(gen, tokens, nkv, hd, unit, spread):
    """A pool [tokens, nkv * hd] of e4m3 values and its scales [tokens / unit, nkv]."""
    x = torch.randn((tokens // unit, unit, nkv, hd), generator=gen, device=DEVICE)
    x *= torch.exp(spread * torch.randn((tokens // unit, 1, nkv, 1), generator=gen, device=DEVICE))
    scale = _pow2_scale(torch.maximum(x.amax((1, 3)), -x.amin((1, 3))))
    x /= scale[:, None, :, None]
    return x.to(EIGHT).view(tokens, nkv * hd), scale


def _tables(r, need, slack=0):
    """Page tables of sequences that need so many pages, pages shuffled; the pool's size, the pages left over."""
    table_len = max(1, int(need.max()) + slack)
    pages = int(need.sum()) + 3
    order = r.permutation(pages)
    table = np.zeros((len(need), table_len), np.int32)
    at = 0
    for i, p in enumerate(need):
        table[i, :p] = order[at:at + p]
        at += int(p)
    return table, pages, table_len, order[at:]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    ctx, rows = _shapes(case)
    kv = ctx + rows
    total = int(rows.sum())
    start = np.concatenate([[0], np.cumsum(rows)])
    s = dict(case=case, op=case["op"], n=case["n"], page=case["page"], ctx=_int32(ctx), rows=total,
             status=torch.zeros(2, dtype=torch.int32, device=DEVICE))

    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=DEVICE)

    if case["op"] == "plan":
        held = _held(case)
        need = -(-kv // case["page"])
        spare = int(np.maximum(need - held, 0).sum())
        most = np.maximum(held, need)
        table_len = max(1, int(most.max()))
        pages = int(held.sum()) + spare + 5
        order = r.permutation(pages).astype(np.int32)
        table = np.full((case["n"], table_len), -1, np.int32)
        at = 0
        for i, p in enumerate(held):
            table[i, :p] = order[at:at + p]
            at += int(p)
        free = np.full(pages, -1, np.int32)
        free[:pages - at] = order[at:]
        s.update(new_rows=_int32(rows), table=_int32(table), table_len=table_len, pages=pages, held=_int32(held), free=_int32(free),
                 n_free=_int32([pages - at]), max_rows=total + 3, held_out=ints(case["n"]), n_free_out=ints(1),
                 row_start=ints(case["n"] + 1), slot=ints(total + 3), pos=ints(total + 3), row_seq=ints(total + 3))
        return s
    nq, nkv, hd, unit = case["nq"], case["nkv"], case["hd"], case["unit"]
    table, pages, table_len, _ = _tables(r, -(-kv // case["page"]))
    s.update(nq=nq, nkv=nkv, hd=hd, unit=unit, table=_int32(table), pages=pages, table_len=table_len, start=_int32(start))
    if case["op"] == "write":
        # one projection's rows: query heads, key heads, value heads
        x = _normal(gen, (total, (nq + 2 * nkv) * hd), 2.0)
        longest = int(kv.max()) + 1
        angle = torch.arange(longest, device=DEVICE, dtype=torch.float64)[:, None] * \
            1e7 ** (-torch.arange(32, device=DEVICE, dtype=torch.float64) / 32)
        angle = torch.cat([angle, angle], 1)
        s.update(x=x, stride=(nq + 2 * nkv) * hd, q=x[:, :nq * hd], k=x[:, nq * hd:(nq + nkv) * hd], v=x[:, (nq + nkv) * hd:],
                 q_w=_normal(gen, (hd,), 0.1), k_w=_normal(gen, (hd,), 0.1), eps=1e-6, cos=torch.cos(angle).to(torch.bfloat16),
                 sin=torch.sin(angle).to(torch.bfloat16), longest=longest, held=case["held"],
                 q_out=torch.zeros((total, nq * hd), dtype=torch.bfloat16, device=DEVICE))
        tokens = pages * case["page"]
        if case["held"] == 8:
            s["k_pool"], s["k_scale"] = _pool_8(gen, tokens, nkv, hd, unit, 0.3)
            s["v_pool"], s["v_scale"] = _pool_8(gen, tokens, nkv, hd, unit, 0.3)
        else:
            s.update(k_pool=_normal(gen, (tokens, nkv * hd)), v_pool=_normal(gen, (tokens, nkv * hd)), k_scale=None, v_scale=None)
        return s
    tokens = pages * case["page"]
    s["k_pool"], s["k_scale"] = _pool_8(gen, tokens, nkv, hd, unit, 0.1)
    s["v_pool"], s["v_scale"] = _pool_8(gen, tokens, nkv, hd, unit, 0.5)
    words = (int(rows.max()) + 31) // 32 if case["mask"] == "tree" else 0
    s.update(most=int(rows.max()), cols=int(kv.max()), words=words, scale=hd ** -0.5, first=case["first"], window=case["window"],
             bits=_int32(_tree_bits(r, rows, words).view(np.int32)) if words else None, q=_normal(gen, (total, nq * hd), 1.5),
             out=torch.zeros((total, nq * hd), dtype=torch.bfloat16, device=DEVICE),
             lse=torch.zeros((total, nq), dtype=torch.float32, device=DEVICE))
    return s


# ---------------------------------------------------------------- plain forms

def _row_of(start, rows):
    """Sequence and index in it of each row."""
    row = torch.arange(rows, device=DEVICE)
    seq = torch.searchsorted(start.long(), row, right=True) - 1
    return seq, row - start.long()[seq]


def _plain_plan(s):
    ctx, new, held, page = s["ctx"].long(), s["new_rows"].long(), s["held"].long(), s["page"]
    need = (ctx + new + page - 1) // page
    back, take = torch.clamp(held - need, min=0), torch.clamp(need - held, min=0)
    at = torch.arange(s["table_len"], device=DEVICE)[None]
    n_free = s["n_free"].long()
    returned = (at >= need[:, None]) & (at < held[:, None])  # in sequence order, ascending within a sequence
    seq, i = returned.nonzero(as_tuple=True)
    s["free"][n_free + torch.arange(seq.numel(), device=DEVICE)] = s["table"][seq, i]
    height = n_free + back.sum()
    taken = (at >= held[:, None]) & (at < need[:, None])
    seq, i = taken.nonzero(as_tuple=True)
    s["table"][seq, i] = s["free"][height - 1 - torch.arange(seq.numel(), device=DEVICE)]
    s["held_out"].copy_(need)
    s["n_free_out"].copy_(height - take.sum())
    s["row_start"][1:] = torch.cumsum(new, 0)
    row = torch.arange(s["max_rows"], device=DEVICE)
    seq = torch.searchsorted(s["row_start"].long(), row, right=True) - 1
    there = row < s["row_start"][-1]
    seq = torch.where(there, seq, torch.zeros_like(seq))
    t = torch.where(there, ctx[seq] + row - s["row_start"].long()[seq], torch.zeros_like(row))
    s["slot"].copy_(torch.where(there, s["table"][seq, t // page].long() * page + t % page, torch.full_like(row, -1)))
    s["pos"].copy_(t)
    s["row_seq"].copy_(torch.where(there, seq, torch.full_like(seq, -1)))
    return _plan_out(s)


def _plan_out(s):
    return {k: s[k] for k in ("table", "held_out", "free", "n_free_out", "row_start", "slot", "pos", "row_seq")}


def _prepared(x, w, cos, sin, eps):
    """(1 + w) RMSNorm of heads [rows, heads, hd], then the rotation of the first 64 dims."""
    x = x.double()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (1.0 + w.double())
    a, b, rest = x[..., :32], x[..., 32:64], x[..., 64:]
    c, n = cos.double()[:, None, :32], sin.double()[:, None, :32]
    return torch.cat([a * c - b * n, b * c + a * n, rest], -1)


def _into_8(s, pool, scale, x, seq, tok, slot):
    """x [rows, nkv, hd] at their slots; a block that is partly full keeps its scale or moves to a larger one."""
    nkv, hd, unit = s["nkv"], s["hd"], s["unit"]
    ctx = s["ctx"].long()
    block = slot // unit
    need = torch.zeros((scale.shape[0], nkv), dtype=torch.float32, device=DEVICE)
    need.scatter_reduce_(0, block[:, None].expand(-1, nkv), x.abs().amax(-1).float(), "amax")
    # sequences that add to a block that they had begun
    count = torch.zeros(s["n"], dtype=torch.long, device=DEVICE).scatter_add_(0, seq, torch.ones_like(seq))
    begun = (ctx % unit != 0) & (count > 0)
    t0 = torch.where(begun, ctx, torch.zeros_like(ctx))
    first = s["table"].long()[torch.arange(s["n"], device=DEVICE), t0 // s["page"]] * s["page"] + t0 % s["page"]
    first = first // unit
    kept = torch.zeros_like(scale)
    kept[first[begun]] = scale[first[begun]]
    new = torch.maximum(_pow2_scale(need), kept)
    j = torch.arange(unit, device=DEVICE)[None]
    old = begun[:, None] & (j < (ctx % unit)[:, None])
    who, at = old.nonzero(as_tuple=True)
    where = first[who] * unit + at
    held = pool.view(-1, nkv, hd)
    again = held[where].float() * scale[first[who]][..., None]
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEVICE)
    touched[block] = True
    scale.copy_(torch.where(touched[:, None], new, scale))
    held[where] = _over(again, scale[first[who]][..., None]).to(EIGHT)
    held[slot] = _over(x, scale[block][..., None].to(x.dtype)).to(EIGHT)


def _plain_write(s):
    nq, nkv, hd, page = s["nq"], s["nkv"], s["hd"], s["page"]
    seq, j = _row_of(s["start"], s["rows"])
    tok = s["ctx"].long()[seq] + j
    slot = s["table"].long()[seq, tok // page] * page + tok % page
    cos, sin = s["cos"][tok], s["sin"][tok]
    s["q_out"].copy_(_prepared(s["q"].reshape(-1, nq, hd), s["q_w"], cos, sin, s["eps"]).view(-1, nq * hd))
    k = _prepared(s["k"].reshape(-1, nkv, hd), s["k_w"], cos, sin, s["eps"])
    v = s["v"].reshape(-1, nkv, hd)
    if s["held"] == 16:
        s["k_pool"][slot] = k.view(-1, nkv * hd).to(torch.bfloat16)
        s["v_pool"][slot] = v.reshape(-1, nkv * hd)
        return _write_out(s)
    _into_8(s, s["k_pool"], s["k_scale"], k.float(), seq, tok, slot)
    _into_8(s, s["v_pool"], s["v_scale"], v.float(), seq, tok, slot)
    return _write_out(s)


def _write_out(s):
    return {k: s[k] for k in ("q_out", "k_pool", "v_pool", "k_scale", "v_scale") if s[k] is not None}


def _plain_attend(s):
    n, most, nkv, hd, cols = s["n"], s["most"], s["nkv"], s["hd"], s["cols"]
    group, page = s["nq"] // nkv, s["page"]
    seq, j = _row_of(s["start"], s["rows"])

    def padded(x):
        y = x.new_zeros((n, most) + x.shape[1:])
        y[seq, j] = x
        return y

    t = torch.arange(cols, device=DEVICE)
    slots = s["table"].long()[:, torch.clamp(t // page, max=s["table_len"] - 1)] * page + t % page

    def held(pool, scale):
        return pool.view(-1, nkv, hd)[slots].float() * scale[slots // s["unit"]][..., None]

    q = padded(s["q"].float()).view(n, most, nkv, group, hd).permute(0, 2, 1, 3, 4).reshape(n, nkv, -1, hd)
    logits = torch.matmul(q, held(s["k_pool"], s["k_scale"]).permute(0, 2, 3, 1)) * s["scale"]
    # [n, most, cols]: which tokens a row sees
    ctx = s["ctx"].long()[:, None, None]
    count = (s["start"][1:] - s["start"][:-1]).long()[:, None, None]
    drafted = t[None, None, :] - ctx
    at = torch.arange(most, device=DEVICE)[None, :, None]
    if s["bits"] is None:
        depth, sees = at, drafted <= at
    else:
        words = padded(s["bits"])
        k = torch.arange(32 * s["words"], device=DEVICE)
        bit = ((words[:, :, k // 32] >> (k % 32).int()) & 1).bool() & (k[None, None] < count)
        depth = torch.clamp(bit.sum(-1, keepdim=True) - 1, min=0)
        sees = (drafted < 0) | torch.gather(bit, 2, torch.clamp(drafted, 0, 32 * s["words"] - 1).expand(-1, most, -1))
    if s["window"]:
        near = (t < s["first"]) | (ctx + depth - t < s["window"])
        sees = sees & (near if s["bits"] is None else near | (drafted >= 0))
    sees = sees & (drafted < count) & (at < count)
    logits = logits.masked_fill(~sees.repeat_interleave(group, 1)[:, None], -math.inf)
    top = torch.clamp(logits.amax(-1, keepdim=True), min=-3e38)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, held(s["v_pool"], s["v_scale"]).permute(0, 2, 1, 3))
    out = out / torch.where(total == 0, torch.ones_like(total), total)

    def rows(x):  # [n, nkv, most * group, d] -> [rows, nq * d]
        return x.view(n, nkv, most, -1, x.shape[-1]).transpose(1, 2)[seq, j].reshape(s["rows"], -1)

    s["out"].copy_(rows(out))
    s["lse"].copy_(rows(top + torch.log(total)))
    return dict(out=s["out"], lse=s["lse"])


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import sparse_attention_token_qsa_gb300 as qsa

    if s["op"] == "plan":
        qsa.qsa_page_plan(s["ctx"], s["new_rows"], s["n"], s["page"], s["pages"], s["table"], s["table_len"], s["table_len"],
                          s["held"], s["held_out"], s["free"], s["n_free"], s["n_free_out"], s["max_rows"], s["row_start"],
                          s["slot"], s["pos"], s["row_seq"], s["status"])
        return _plan_out(s)
    if s["op"] == "write":
        qsa.qsa_qkv_write(s["q"], s["stride"], s["nq"], s["k"], s["stride"], s["v"], s["stride"], s["nkv"], s["hd"], s["q_w"],
                          s["k_w"], s["eps"], s["cos"], s["sin"], s["longest"], None, s["ctx"], s["start"], s["n"], s["rows"],
                          s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["unit"], s["pages"], s["page"], s["table"],
                          s["table_len"], s["table_len"], s["q_out"], s["nq"] * s["hd"], s["status"])
        return _write_out(s)
    d = s["nq"] * s["hd"]
    if "workspace" not in s:  # a program makes it once
        s["workspace"] = qsa.new_cache8_workspace(s["n"], s["rows"], s["nq"], s["nkv"], s["hd"])
    qsa.qsa_cache8_attn(s["q"], d, s["nq"], s["nkv"], s["hd"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["unit"],
                        s["pages"], s["page"], s["table"], s["table_len"], s["table_len"], s["ctx"], s["start"], s["n"], s["rows"],
                        s["bits"], s["words"], s["first"], s["window"], s["scale"], s["out"], d, s["lse"], s["status"],
                        s["workspace"])
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "write": _plain_write, "attend": _plain_attend}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits

def _slots_of(s, i, t):
    """Pool rows of tokens t (a tensor) of sequence i."""
    return s["table"][i].long()[t // s["page"]] * s["page"] + t % s["page"]


def _exact_write(s):
    nq, nkv, hd, unit = s["nq"], s["nkv"], s["hd"], s["unit"]
    if s["k_pool"].numel() > 1 << 28:
        return None
    got = {k: s[k].double() for k in ("q_out", "k_pool", "v_pool", "k_scale", "v_scale") if s[k] is not None}
    start, ctx = s["start"].tolist(), s["ctx"].tolist()
    for i in range(s["n"]):
        a, b, c = start[i], start[i + 1], ctx[i]
        if a == b:
            continue
        tok = torch.arange(c, c + b - a, device=DEVICE)
        turn = torch.complex(s["cos"][tok, :32].double(), s["sin"][tok, :32].double())[:, None]
        ready = {}
        for name, heads, w in (("q", nq, s["q_w"]), ("k", nkv, s["k_w"])):
            x = s[name][a:b].double().reshape(-1, heads, hd)
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + s["eps"]) * (w.double() + 1)
            z = torch.complex(x[..., :32], x[..., 32:64]) * turn
            ready[name] = torch.cat([z.real, z.imag, x[..., 64:]], -1)
        ready["v"] = s["v"][a:b].double().reshape(-1, nkv, hd)
        got["q_out"][a:b] = ready["q"].reshape(b - a, -1)
        slots = _slots_of(s, i, tok)
        for name in ("k", "v"):
            if s["held"] == 16:
                got[name + "_pool"][slots] = ready[name].reshape(b - a, -1)
                continue
            pool, scale = got[name + "_pool"].view(-1, nkv, hd), got[name + "_scale"]
            amax = ready[name].abs().amax(-1)
            for u in range(c // unit, (c + b - a - 1) // unit + 1):
                lo, hi = max(c, u * unit), min(c + b - a, (u + 1) * unit)
                need = amax[lo - c:hi - c].amax(0)
                blk = int(slots[lo - c]) // unit
                want = torch.exp2(torch.round(torch.log2(torch.clamp(need, min=1e-30) / MOST_8)))  # or one of its neighbours
                want = torch.where(want * MOST_8 < need, 2 * want, torch.where(want * MOST_8 / 2 >= need, want / 2, want)) * (need > 0)
                if lo > u * unit:
                    old = scale[blk].clone()
                    want = torch.maximum(want, old)
                    rows = torch.arange(blk * unit, blk * unit + lo - u * unit, device=DEVICE)
                    pool[rows] = pool[rows] * (old / torch.clamp(want, min=1e-300))[None, :, None]
                scale[blk] = want
                pool[slots[lo - c:hi - c]] = ready[name][lo - c:hi - c] / torch.clamp(want, min=1e-300)[None, :, None]
    return got


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s)
    start, ctx = s["start"].tolist(), s["ctx"].tolist()
    group, hd, unit = s["nq"] // s["nkv"], s["hd"], s["unit"]
    out = torch.zeros((s["rows"], s["nq"] * hd), dtype=torch.float64, device=DEVICE)
    lses = torch.zeros((s["rows"], s["nq"]), dtype=torch.float64, device=DEVICE)
    for i in range(s["n"]):
        a, b, c = start[i], start[i + 1], ctx[i]
        kv = c + b - a
        at = _slots_of(s, i, torch.arange(kv, device=DEVICE))
        t = torch.arange(kv, device=DEVICE)[None]
        r = torch.arange(b - a, device=DEVICE)[:, None]
        vis = torch.ones((b - a, kv), dtype=torch.bool, device=DEVICE)
        depth = r
        if s["bits"] is None:
            vis = t <= c + r
        else:
            for k in range(b - a):  # drafted token k, seen by each row
                vis[:, c + k] = (s["bits"][a:b, k // 32] >> (k % 32)) & 1 == 1
            depth = torch.clamp(vis[:, c:].sum(1, keepdim=True) - 1, min=0)
        if s["window"]:
            far = (t >= s["first"]) & (c + depth - t >= s["window"])
            if s["bits"] is not None:
                far = far & (t < c)
            vis = vis & ~far
        for h in range(s["nkv"]):
            key = s["k_pool"][at][:, h * hd:(h + 1) * hd].double() * s["k_scale"][at // unit, h].double()[:, None]
            val = s["v_pool"][at][:, h * hd:(h + 1) * hd].double() * s["v_scale"][at // unit, h].double()[:, None]
            for head in range(h * group, (h + 1) * group):
                x = (s["q"][a:b, head * hd:(head + 1) * hd].double() @ key.T) * s["scale"]
                x[~vis] = -math.inf
                lse = torch.logsumexp(x, 1)
                lses[a:b, head] = lse
                out[a:b, head * hd:(head + 1) * hd] = torch.nan_to_num(torch.exp(x - lse[:, None])) @ val
    return dict(out=out, lse=lses)
