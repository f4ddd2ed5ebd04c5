"""Cases of the cache operators: tree attention over a paged K/V cache, the attention weight its
tokens gather, the choice of the tokens a shortened cache keeps, and the move that shortens it.

With ``own`` false ``run`` computes each operator from elementary torch operations in 32 bits;
with ``own`` true it calls the library.  ``exact`` computes the same results in 64 bits, one
sequence at a time.  Lengths and drafted counts follow from a case alone, contents from the seed.
"""
import functools
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


def listed():
    return [
        # --- attention of drafted rows over every cached token
        # one sequence early in its answer, one token at a time: latency is all
        dict(name="tree one row 515", op="tree", n=1, lo=515, hi=515, rlo=1, rhi=1, nq=16, nkv=2,
             hd=256, page=16, mask="chain", shape=1),
        # a decode batch without drafts: every sequence's whole cache read for one row
        dict(name="tree decode 16x64k", op="tree", n=16, lo=16384, hi=65535, rlo=1, rhi=1, nq=16,
             nkv=2, hd=256, page=16, mask="chain", shape=2),
        # one long sequence verifying a tree of 64 drafted tokens
        dict(name="tree verify 64 of 64k", op="tree", n=1, lo=65471, hi=65471, rlo=64, rhi=64, nq=16,
             nkv=2, hd=256, page=16, mask="tree", shape=3),
        # a serving batch verifying small trees of odd sizes over short and middle contexts
        dict(name="tree verify batch", op="tree", n=24, lo=300, hi=9001, rlo=5, rhi=37, nq=32, nkv=8,
             hd=128, page=64, mask="tree", shape=4),
        # wide trees: the products are what costs
        dict(name="tree wide 4x128", op="tree", n=4, lo=7000, hi=16001, rlo=127, rhi=128, nq=32,
             nkv=8, hd=128, page=16, mask="tree", shape=5),
        # --- the attention weight that cached tokens gather
        dict(name="mass one row 515", op="mass", n=1, lo=515, hi=515, rlo=1, rhi=1, nq=16, nkv=2,
             hd=256, page=16, mask="chain", shape=6, carry=1.0),
        # the decode batch again: each step adds its row's weights
        dict(name="mass decode 16x64k", op="mass", n=16, lo=16384, hi=65535, rlo=1, rhi=1, nq=16,
             nkv=2, hd=256, page=16, mask="chain", shape=7, carry=1.0),
        # a window of 64 rows at the end of a long prompt decides what stays
        dict(name="mass window 64 of 64k", op="mass", n=1, lo=65471, hi=65471, rlo=64, rhi=64, nq=16,
             nkv=2, hd=256, page=16, mask="tree", shape=8, carry=0.5),
        # --- which tokens stay
        # one sequence just past its budget, whole 4-token blocks
        dict(name="evict one of 4099", op="evict", n=1, lo=4099, hi=4099, nkv=2, keep=2048, first=4,
             last=128, unit=4, shape=9),
        # long caches cut back to 8192 tokens
        dict(name="evict 32x262k", op="evict", n=32, lo=131072, hi=262144, nkv=2, keep=8192, first=16,
             last=1024, unit=4, shape=10),
        # --- the move
        # accepted drafted tokens join their contexts: a few rows a sequence
        dict(name="compact accepted 24", op="compact", n=24, lo=300, hi=9001, rlo=5, rhi=37, nkv=8,
             hd=128, page=64, unit=0, keep=0, shape=11),
        # caches cut back to 8192 tokens, blocks' pooled keys and weights with them
        dict(name="compact 16x64k", op="compact", n=16, lo=16384, hi=65535, nkv=2, hd=256, page=16,
             unit=4, keep=8192, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "mass", "mass", "evict", "compact"])
    nq, nkv, hd = rng.choice([(16, 2, 256), (32, 8, 128), (8, 1, 128), (24, 2, 256), (6, 2, 128),
                              (12, 4, 256)])
    n = _log_int(rng, 1, 40)
    c = dict(op=op, n=n, nkv=nkv, shape=rng.randrange(1 << 30))
    if op == "evict":
        unit = rng.choice([1, 4])
        hi = _log_int(rng, 64, min(262144, 8000000 // (n * nkv)))
        lo = max(32, hi // rng.randint(1, 4))
        keep = unit * max(1, _log_int(rng, 8, lo - 4) // unit)
        first = unit * rng.randint(0, keep // (4 * unit))
        last = unit * rng.randint(0, keep // (2 * unit))
        return dict(c, lo=lo, hi=hi, keep=keep, first=first, last=last,
                    unit=unit)
    width = nkv * hd
    hi = _log_int(rng, 1, max(2, min(65536, 1000000000 // (n * width * 4))))
    lo = max(0, hi // rng.randint(1, 8) - 1)
    c.update(hd=hd, lo=lo, hi=hi, page=rng.choice([1, 7, 16, 16, 32, 64, 100, 256]))
    if op == "compact":
        unit = rng.choice([0, 1, 4])
        rhi = rng.randint(2, 48)
        return dict(c, unit=unit, rlo=rng.randint(1, rhi), rhi=rhi,
                    keep=0 if unit == 0 else unit * max(1, _log_int(rng, 4, max(5, hi)) // unit))
    rows_most = max(1, min(128, int(5e10 / (4.0 * n * nq * hd * (hi + 128)))))
    rhi = _log_int(rng, 1, rows_most)
    c.update(nq=nq, rlo=rng.randint(1, rhi), rhi=rhi, mask=rng.choice(["tree", "tree", "chain"]))
    if op == "mass":
        c["carry"] = rng.choice([1.0, 0.5, 0.0])
    return c


# ---------------------------------------------------------------- shapes and inputs

def _shapes(case):
    """Cached lengths and drafted counts of a case: numpy int arrays."""
    r = np.random.RandomState(case["shape"] % (1 << 31))
    ctx = r.randint(case["lo"], case["hi"] + 1, size=case["n"]).astype(np.int64)
    if "rlo" not in case or case.get("unit", 0):
        return ctx, np.zeros(case["n"], np.int64)
    return ctx, r.randint(case["rlo"], case["rhi"] + 1, size=case["n"]).astype(np.int64)


def work(case):
    ctx, rows = _shapes(case)
    kv = ctx + rows
    if case["op"] in ("tree", "mass"):
        per = case["nkv"] * case["hd"] * 2
        q = int(rows.sum()) * case["nq"] * case["hd"] * 2
        lse = int(rows.sum()) * case["nq"] * 4
        pairs = int((rows * ctx).sum() + (rows * (rows + 1) // 2).sum())
        if case["op"] == "tree":
            return dict(bytes=2 * per * int(kv.sum()) + 2 * q + lse,
                        flops=4 * pairs * case["nq"] * case["hd"])
        return dict(bytes=per * int(kv.sum()) + q + lse + 8 * case["nkv"] * int(kv.sum()),
                    flops=2 * pairs * case["nq"] * case["hd"])
    if case["op"] == "evict":
        return dict(bytes=4 * case["nkv"] * int(ctx.sum()) + 4 * int(np.minimum(ctx, case["keep"]).sum()),
                    flops=case["nkv"] * int(ctx.sum()))
    if case["unit"] == 0:
        moved = int(((rows + 1) // 2).sum())
    else:
        moved = int(np.minimum(ctx, case["keep"]).sum())
    a_token = 8 * case["nkv"] * case["hd"] + 8 * case["nkv"] + (128 if case["unit"] == 4 else 0)
    return dict(bytes=moved * (a_token + 4), flops=0)


def _tree_bits(r, rows, words, mask):
    """Which drafted tokens each drafted row sees, itself among them: uint32 words [sum(rows), words]."""
    n, most = len(rows), int(rows.max())
    sees = np.zeros((n, most, most), bool)
    for k in range(most):  # a token's parent is an earlier one, or the context (-1)
        if k:
            parent = np.maximum(-1, k - 1 - r.geometric(0.4, size=n) + 1)
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


def _paged(gen, r, kv, page, width, planes):
    """`planes` pools [pages * page, width] and the sequences' page tables, pages shuffled."""
    per = (kv + page - 1) // page
    table_len = max(1, int(per.max()))
    pages = int(per.sum()) + 3
    order = r.permutation(pages)
    table = np.zeros((len(kv), table_len), np.int32)
    at = 0
    for i, p in enumerate(per):
        table[i, :p] = order[at:at + p]
        at += int(p)
    pools = [_normal(gen, (pages * page, width)) for _ in range(planes)]
    return pools, table, pages, table_len


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    ctx, rows = _shapes(case)
    kv = ctx + rows
    s = dict(case=case, op=case["op"], n=case["n"], nkv=case["nkv"], status=torch.zeros(2, dtype=torch.int32, device=DEVICE))
    if case["op"] == "evict":
        # most of the weight sits on few tokens; a token no row attended has none
        cols = (case["hi"] + 3) // 4 * 4
        u = torch.rand((case["n"], case["nkv"], cols), generator=gen, device=DEVICE)
        mass = torch.where(u < 0.3, torch.zeros_like(u), u.pow(12.0) * 8.0)
        s.update(mass=mass, cols=cols, tokens=case["hi"], length=_int32(ctx), keep=case["keep"], first=case["first"],
                 last=case["last"], unit=case["unit"], sel_cols=case["keep"] + case["unit"] - 1)
        s["sel"] = torch.full((case["n"], s["sel_cols"]), -1, dtype=torch.int32, device=DEVICE)
        s["n_sel"] = torch.zeros(case["n"], dtype=torch.int32, device=DEVICE)
        return s
    width = case["nkv"] * case["hd"]
    (k_pool, *more), table, pages, table_len = _paged(gen, r, kv, case["page"], width, 1 if case["op"] == "mass" else 2)
    s.update(k_pool=k_pool, table=_int32(table), pages=pages, table_len=table_len, page=case["page"], ctx=_int32(ctx),
             hd=case["hd"], cols=max(4, (int(kv.max()) + 3) // 4 * 4))
    if more:
        s["v_pool"] = more[0]
    if case["op"] == "compact":
        s.update(unit=case["unit"], width=width)
        lists = []
        for i in range(case["n"]):
            if case["unit"] == 0:  # the accepted tokens: a random half of the drafted ones, in order
                lists.append(ctx[i] + np.sort(r.permutation(rows[i])[:(rows[i] + 1) // 2]))
                continue
            unit, units = case["unit"], int(ctx[i]) // case["unit"]
            stay = np.sort(r.permutation(units)[:case["keep"] // unit])
            lists.append(np.concatenate([(stay[:, None] * unit + np.arange(unit)).reshape(-1),
                                         np.arange(units * unit, ctx[i])]))
        s["max_keep"] = max(1, max(len(x) for x in lists))
        keep = np.full((case["n"], s["max_keep"]), -1, np.int64)
        for i, x in enumerate(lists):
            keep[i, :len(x)] = x
        s.update(keep=_int32(keep), n_keep=_int32([len(x) for x in lists]),
                 base=_int32(ctx if case["unit"] == 0 else 0 * ctx))
        s["mass"] = torch.rand((case["n"], case["nkv"], s["cols"]), generator=gen, device=DEVICE)
        if case["unit"] == 4:
            per = s["cols"] // 4
            s["block_keys"] = _normal(gen, (case["n"] * per, 128))
            s["key_base"] = torch.arange(case["n"], dtype=torch.int64, device=DEVICE) * per
        return s
    start = np.concatenate([[0], np.cumsum(rows)])
    words = (int(rows.max()) + 31) // 32
    s.update(start=_int32(start), rows=int(start[-1]), most=int(rows.max()), nq=case["nq"], words=words,
             scale=case["hd"] ** -0.5,
             bits=_int32(_tree_bits(r, rows, words, case["mask"]).view(np.int32)) if case["mask"] == "tree" else None)
    s["q"] = _normal(gen, (s["rows"], case["nq"] * case["hd"]), 1.5)
    s["lse"] = torch.zeros((s["rows"], case["nq"]), dtype=torch.float32, device=DEVICE)
    if case["op"] == "tree":
        s["out"] = torch.zeros((s["rows"], case["nq"] * case["hd"]), dtype=torch.bfloat16, device=DEVICE)
        return s
    logits, sees, _ = _logits(s)
    lse = torch.logsumexp(logits.masked_fill(~sees, -math.inf).double(), -1).float()
    s["lse"].copy_(_rows_from_padded(s, lse[..., None]).reshape(s["rows"], s["nq"]))
    s["weight"] = (torch.rand(s["rows"], generator=gen, device=DEVICE) < 0.75).float() if case["mask"] == "tree" else None
    s["carry"] = case["carry"]
    s["mass"] = torch.rand((case["n"], case["nkv"], s["cols"]), generator=gen, device=DEVICE)
    return s


# ---------------------------------------------------------------- plain forms

def _row_of(s):
    """Sequence and drafted index of each row."""
    start = s["start"].long()
    row = torch.arange(s["rows"], device=DEVICE)
    seq = torch.searchsorted(start, row, right=True) - 1
    return seq, row - start[seq]


def _slots(s, most):
    """Pool row of token t of each sequence (tokens past a table's end: row 0)."""
    t = torch.arange(most, device=DEVICE)
    page = torch.clamp(t // s["page"], max=s["table_len"] - 1)
    return s["table"].long()[:, page] * s["page"] + t % s["page"]


def _padded_rows(s, x):
    """[rows, ...] -> [n, most, ...], zeros past a sequence's rows."""
    seq, j = _row_of(s)
    y = x.new_zeros((s["n"], s["most"]) + x.shape[1:])
    y[seq, j] = x
    return y


def _rows_from_padded(s, x):
    """[n, nkv, most * group, d] -> [rows, nq * d]"""
    seq, j = _row_of(s)
    n, nkv, _, d = x.shape
    return x.view(n, nkv, s["most"], -1, d).transpose(1, 2)[seq, j].reshape(s["rows"], -1)


def _logits(s):
    """Scaled logits [n, nkv, most * group, kv], which of them a row sees, and the padded slots."""
    group, most_kv = s["nq"] // s["nkv"], s["cols"]
    slots = _slots(s, most_kv)
    keys = s["k_pool"].view(-1, s["nkv"], s["hd"])[slots].float().permute(0, 2, 3, 1)
    q = _padded_rows(s, s["q"].float()).view(s["n"], s["most"], s["nkv"], group, s["hd"])
    q = q.permute(0, 2, 1, 3, 4).reshape(s["n"], s["nkv"], -1, s["hd"])
    logits = torch.matmul(q, keys) * s["scale"]
    t = torch.arange(most_kv, device=DEVICE)
    drafted = t[None, None, :] - s["ctx"].long()[:, None, None]  # [n, 1, kv]
    count = (s["start"][1:] - s["start"][:-1]).long()[:, None, None]
    if s["bits"] is None:
        sees = drafted <= torch.arange(s["most"], device=DEVICE)[None, :, None]
    else:
        words = _padded_rows(s, s["bits"])
        k = torch.clamp(drafted, 0, 32 * s["words"] - 1).expand(-1, s["most"], -1)
        bit = (torch.gather(words, 2, k // 32) >> (k % 32).int()) & 1
        sees = (drafted < 0) | (bit != 0)
    j = torch.arange(s["most"], device=DEVICE)[None, :, None]
    sees = sees & (drafted < count) & (j < count)  # rows past a sequence's own see nothing
    return logits, sees.repeat_interleave(group, 1)[:, None], slots


def _plain_tree(s):
    logits, sees, slots = _logits(s)
    logits = logits.masked_fill(~sees, -math.inf)
    top = torch.clamp(logits.amax(-1, keepdim=True), min=-3e38)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    values = s["v_pool"].view(-1, s["nkv"], s["hd"])[slots].float().permute(0, 2, 1, 3)
    out = torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(_rows_from_padded(s, out))
    s["lse"].copy_(_rows_from_padded(s, top + torch.log(total)))
    return dict(out=s["out"], lse=s["lse"])


def _plain_mass(s):
    logits, sees, _ = _logits(s)
    group = s["nq"] // s["nkv"]
    lse = _padded_rows(s, s["lse"]).view(s["n"], s["most"], s["nkv"], group).transpose(1, 2).reshape(s["n"], s["nkv"], -1, 1)
    p = torch.where(sees, torch.exp(logits - lse), torch.zeros_like(logits))
    if s["weight"] is not None:
        w = _padded_rows(s, s["weight"]).repeat_interleave(group, 1)
        p = p * w[:, None, :, None]
    t = torch.arange(s["cols"], device=DEVICE)
    ctx = s["ctx"].long()[:, None]
    kv = ctx + (s["start"][1:] - s["start"][:-1]).long()[:, None]
    old = torch.where((t < ctx)[:, None], s["mass"] * s["carry"], torch.zeros_like(s["mass"]))
    s["mass"].copy_(torch.where((t < kv)[:, None], old + p.sum(2), s["mass"]))
    return dict(mass=s["mass"])


def _plain_evict(s):
    unit, most = s["unit"], s["cols"] // s["unit"]
    token = functools.reduce(torch.add, s["mass"].unbind(1))  # heads in order
    score = functools.reduce(torch.add, token.view(s["n"], most, unit).unbind(2))  # tokens in order
    units = (s["length"].long() // unit)[:, None]
    u = torch.arange(most, device=DEVICE)[None]
    score = torch.where((u < s["first"] // unit) | (u >= units - s["last"] // unit), torch.full_like(score, math.inf), score)
    score = torch.where(u < units, score, torch.full_like(score, -math.inf))
    order = torch.sort(score, dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order[:, :s["keep"] // unit], True) & (u < units)
    t = torch.arange(most * unit, device=DEVICE)[None]
    length = s["length"].long()[:, None]
    stays = (kept.repeat_interleave(unit, 1) | (t >= units * unit)) & (t < length)
    n_sel = stays.sum(1)
    at = torch.cumsum(stays, 1) - 1
    seq, tok = stays.nonzero(as_tuple=True)
    s["sel"][seq, at[seq, tok]] = tok.int()
    s["n_sel"].copy_(n_sel)
    return dict(sel=s["sel"], n_sel=s["n_sel"])


def _plain_compact(s):
    j = torch.arange(s["max_keep"], device=DEVICE)[None]
    moves = j < s["n_keep"].long()[:, None]
    seq, at = moves.nonzero(as_tuple=True)
    src, dst = s["keep"].long()[seq, at], s["base"].long()[seq] + at
    table, page = s["table"].long(), s["page"]
    a = table[seq, src // page] * page + src % page
    b = table[seq, dst // page] * page + dst % page
    s["k_pool"][b] = s["k_pool"][a]
    s["v_pool"][b] = s["v_pool"][a]
    s["mass"][seq, :, dst] = s["mass"][seq, :, src]
    out = dict(k_pool=s["k_pool"], v_pool=s["v_pool"], mass=s["mass"])
    if "block_keys" in s:
        whole = (at % 4 == 0) & (at + 4 <= s["n_keep"].long()[seq])
        key_base = s["key_base"][seq[whole]]
        s["block_keys"][key_base + dst[whole] // 4] = s["block_keys"][key_base + src[whole] // 4]
        out["block_keys"] = s["block_keys"]
    return out


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import sparse_attention_token_qsa_gb300 as qsa

    if s["op"] == "tree":
        d = s["nq"] * s["hd"]
        if "workspace" not in s:  # a program makes it once
            s["workspace"] = qsa.new_tree_workspace(s["n"], s["rows"], s["nq"], s["nkv"], s["hd"])
        qsa.qsa_tree_attn(s["q"], d, s["nq"], s["nkv"], s["hd"], s["k_pool"], s["v_pool"], s["pages"], s["page"], s["table"],
                          s["table_len"], s["table_len"], s["ctx"], s["start"], s["n"], s["rows"], s["bits"], s["words"],
                          s["scale"], s["out"], d, s["lse"], s["status"], s["workspace"])
        return dict(out=s["out"], lse=s["lse"])
    if s["op"] == "mass":
        qsa.qsa_attn_mass(s["q"], s["nq"] * s["hd"], s["nq"], s["nkv"], s["hd"], s["k_pool"], s["pages"], s["page"], s["table"],
                          s["table_len"], s["table_len"], s["ctx"], s["start"], s["n"], s["rows"], s["bits"], s["words"],
                          s["scale"], s["lse"], s["weight"], s["carry"], s["mass"], s["cols"], s["status"])
        return dict(mass=s["mass"])
    if s["op"] == "evict":
        qsa.qsa_evict_select(s["mass"], s["cols"], s["nkv"], s["length"], s["n"], s["tokens"], s["keep"], s["first"], s["last"],
                             s["unit"], s["sel"], s["sel_cols"], s["n_sel"], s["status"])
        return dict(sel=s["sel"], n_sel=s["n_sel"])
    qsa.qsa_cache_compact(s["k_pool"], s["v_pool"], s["width"], s["pages"], s["table"], s["table_len"], s["table_len"], s["page"],
                          s["keep"], s["max_keep"], s["n_keep"], s["n"], s["max_keep"], s["base"], s["mass"], s["cols"], s["nkv"],
                          s.get("block_keys"), s.get("key_base"), s["status"])
    out = dict(k_pool=s["k_pool"], v_pool=s["v_pool"], mass=s["mass"])
    if "block_keys" in s:
        out["block_keys"] = s["block_keys"]
    return out


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "mass": _plain_mass, "evict": _plain_evict, "compact": _plain_compact}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "evict":
        return None  # whole numbers
    s = prepare(case, seed)
    start = s["start"].tolist() if "start" in s else None
    ctx, table = s["ctx"].tolist(), s["table"].tolist()

    def rows_of(i, tokens):
        t = torch.as_tensor(tokens, device=DEVICE, dtype=torch.long)
        return torch.as_tensor(table[i], device=DEVICE)[t // s["page"]].long() * s["page"] + t % s["page"]

    if case["op"] == "compact":
        if s["k_pool"].numel() > 1 << 28:
            return None
        got = dict(k_pool=s["k_pool"].double(), v_pool=s["v_pool"].double(), mass=s["mass"].double())
        if "block_keys" in s:
            got["block_keys"] = s["block_keys"].double()
        for i in range(s["n"]):
            m, base = int(s["n_keep"][i]), int(s["base"][i])
            keep = s["keep"][i, :m].long()
            to = torch.arange(base, base + m, device=DEVICE)
            for name in ("k_pool", "v_pool"):
                got[name][rows_of(i, to)] = s[name][rows_of(i, keep)].double()
            got["mass"][i, :, base:base + m] = s["mass"][i][:, keep].double()
            if "block_keys" in s:
                kb = int(s["key_base"][i])
                got["block_keys"][kb:kb + m // 4] = s["block_keys"][kb + keep[0:m // 4 * 4:4] // 4].double()
        return got
    group = s["nq"] // s["nkv"]
    got = dict(out=torch.zeros((s["rows"], s["nq"] * s["hd"]), dtype=torch.float64, device=DEVICE),
               lse=torch.zeros((s["rows"], s["nq"]), dtype=torch.float64, device=DEVICE)) if case["op"] == "tree" else \
        dict(mass=s["mass"].double())
    for i in range(s["n"]):
        a, b = start[i], start[i + 1]
        kv = ctx[i] + b - a
        at = rows_of(i, range(kv)) if kv < 4096 else rows_of(i, torch.arange(kv))
        vis = torch.ones((b - a, kv), dtype=torch.bool, device=DEVICE)
        for k in range(b - a):  # drafted token k, seen by each row
            if s["bits"] is None:
                vis[:, ctx[i] + k] = torch.arange(b - a, device=DEVICE) >= k
            else:
                vis[:, ctx[i] + k] = (s["bits"][a:b, k // 32] >> (k % 32)) & 1 == 1
        for h in range(s["nkv"]):
            key = s["k_pool"][at][:, h * s["hd"]:(h + 1) * s["hd"]].double()
            for g in range(group):
                head = h * group + g
                q = s["q"][a:b, head * s["hd"]:(head + 1) * s["hd"]].double()
                x = (q @ key.T) * s["scale"]
                x[~vis] = -math.inf
                if case["op"] == "tree":
                    val = s["v_pool"][at][:, h * s["hd"]:(h + 1) * s["hd"]].double()
                    lse = torch.logsumexp(x, 1)
                    got["lse"][a:b, head] = lse
                    got["out"][a:b, head * s["hd"]:(head + 1) * s["hd"]] = torch.exp(x - lse[:, None]) @ val
                    continue
                if g == 0:
                    got["mass"][i, h, :ctx[i]] *= s["carry"]
                    got["mass"][i, h, ctx[i]:kv] = 0
                p = torch.exp(x - s["lse"][a:b, head].double()[:, None])
                if s["weight"] is not None:
                    p = p * s["weight"][a:b].double()[:, None]
                got["mass"][i, h, :kv] += p.sum(0)
    return got
