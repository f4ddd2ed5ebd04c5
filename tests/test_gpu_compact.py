"""qsa_cache_compact against numpy's gather and assignment: equal bits everywhere,
moved or not.  Also the four cache operators in turn, as a serving loop uses them."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev, f64, keep_units, ref_tree
from qsa_cases import EPS, THETA

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


class Pool:
    def __init__(self, rng, n, tokens, page, width, nkv, blocks):
        per = -(-tokens // page)
        self.n, self.page, self.width, self.nkv, self.per = n, page, width, nkv, per
        self.pages = n * per + 3
        self.k = qi.paged_kv_pool(rng, self.pages, page, width)
        self.v = qi.paged_kv_pool(rng, self.pages, page, width)
        self.table = rng.permutation(self.pages)[:n * per].reshape(n, per).astype(np.int32)
        self.cols = (tokens + 3) // 4 * 4
        self.mass = rng.random((n, nkv, self.cols), dtype=np.float32)
        self.keys = rng.integers(0, 1 << 16, size=(n * self.cols // 4 + 5, 128), dtype=np.uint16) if blocks else None
        self.base = 2 + np.arange(n, dtype=np.int64) * (self.cols // 4)

    def slots(self, i, t):
        t = np.asarray(t, np.int64)
        return self.table[i, t // self.page].astype(np.int64) * self.page + t % self.page


def call(qsa, p, lists, first, mass=True, max_keep=None, stream=None):
    most = max([len(x) for x in lists] + [1]) if max_keep is None else max_keep
    keep = np.full((p.n, most + 2), -9, np.int32)
    for i, x in enumerate(lists):
        keep[i, :len(x)] = x
    k, v, m, b = dev(p.k), dev(p.v), dev(p.mass), None if p.keys is None else dev(p.keys)
    st = qsa.new_status()
    kd, nd, td = dev(keep), dev(np.array([len(x) for x in lists], np.int32)), dev(p.table)
    fd, bd = None if first is None else dev(np.asarray(first, np.int32)), None if b is None else dev(p.base)
    torch.cuda.synchronize()
    qsa.qsa_cache_compact(k, v, p.width, p.pages, td, p.per, p.per, p.page, kd, most + 2, nd, p.n, most, fd,
                          m if mass else None, p.cols, p.nkv, b, bd, st, stream=stream)
    torch.cuda.synchronize()
    return (k.cpu().numpy().view(np.uint16), v.cpu().numpy().view(np.uint16), m.cpu().numpy(),
            None if b is None else b.cpu().numpy().view(np.uint16), qsa.qsa_read_status(st))


def want(p, lists, first, mass=True):
    k, v, m = p.k.copy(), p.v.copy(), p.mass.copy()
    b = None if p.keys is None else p.keys.copy()
    for i, x in enumerate(lists):
        f = 0 if first is None else int(first[i])
        x = np.asarray(x, np.int64)
        src, dst = p.slots(i, x), p.slots(i, f + np.arange(len(x)))
        k[dst], v[dst] = p.k[src], p.v[src]
        if mass:
            m[i][:, f:f + len(x)] = p.mass[i][:, x]
        if b is not None:
            w = len(x) // 4
            b[p.base[i] + f // 4 + np.arange(w)] = p.keys[p.base[i] + x[0:4 * w:4] // 4]
    return k, v, m, b


def same(got, expect):
    for a, b in zip(got, expect):
        if b is not None:
            assert np.array_equal(a, b)


def whole_blocks(rng, tokens, keep, tail):
    b = np.sort(rng.permutation(tokens // 4)[:keep])
    return np.concatenate([(b[:, None] * 4 + np.arange(4)).reshape(-1), np.arange(tokens // 4 * 4, tokens // 4 * 4 + tail)])


@pytest.mark.parametrize("page,width,nkv", [(16, 512, 2), (1, 8, 1), (7, 1024, 8), (64, 136, 3), (256, 256, 2)])
def test_eviction_lists(qsa, page, width, nkv):
    """Nothing, one token, everything, the front, the back, more than several chunks."""
    rng = qi.rng_for(60, salt=page)
    p = Pool(rng, 7, 5000, page, width, nkv, False)
    some = lambda n: np.sort(rng.permutation(5000)[:n])  # noqa: E731
    lists = [[], [4999], np.arange(5000), np.arange(100), np.arange(4000, 5000), some(2500), some(4990)]
    got = call(qsa, p, lists, None)
    assert got[4] == (0, 0)
    same(got, want(p, lists, None))
    got = call(qsa, p, lists, None, mass=False)
    assert got[4] == (0, 0)
    same(got, want(p, lists, None, mass=False))


def test_blocks_and_tails(qsa):
    rng = qi.rng_for(61)
    p = Pool(rng, 5, 3003, 16, 512, 2, True)
    lists = [whole_blocks(rng, 3003, k, t) for k, t in ((0, 0), (1, 3), (700, 2), (750, 3), (300, 0))]
    got = call(qsa, p, lists, [0] * 5)
    assert got[4] == (0, 0)
    same(got, want(p, lists, [0] * 5))
    first = [4, 8, 0, 0, 600]
    lists = [np.asarray(x)[np.asarray(x) >= 0] + f for x, f in zip([whole_blocks(rng, 2000, 200, 1)] * 5, first)]
    got = call(qsa, p, lists, first)
    assert got[4] == (0, 0)
    same(got, want(p, lists, first))


@pytest.mark.parametrize("page", [1, 16, 50])
def test_accepted_drafts(qsa, page):
    rng = qi.rng_for(62, salt=page)
    p = Pool(rng, 6, 400, page, 1024, 8, False)
    ctx = [0, 1, 15, 200, 363, 399]
    lists = [np.array(x, np.int64) + c for x, c in zip(([0], [0, 3, 7], [], [1, 2, 4, 30], np.arange(36), [0]), ctx)]
    got = call(qsa, p, lists, ctx)
    assert got[4] == (0, 0)
    same(got, want(p, lists, ctx))


def test_lists_in_any_order_and_with_repeats(qsa):
    """Every entry at or past its place: the list is taken as it stands."""
    rng = qi.rng_for(63)
    p = Pool(rng, 2, 4000, 16, 256, 1, False)
    lists = [rng.integers(2000, 4000, size=2000), np.full(1500, 3999)]
    got = call(qsa, p, lists, None)
    assert got[4] == (0, 0)
    same(got, want(p, lists, None))


def test_device_errors(qsa):
    rng = qi.rng_for(64)
    p = Pool(rng, 3, 300, 16, 256, 2, True)
    good = [whole_blocks(rng, 300, 40, 0) for _ in range(3)]
    ok = want(p, good, [0] * 3)

    def others(got):
        for i in (0, 2):
            s = p.slots(i, np.arange(300))
            assert np.array_equal(got[0][s], ok[0][s]) and np.array_equal(got[1][s], ok[1][s])
            assert np.array_equal(got[2][i], ok[2][i])

    for first in ([0, -4, 0], [0, 300, 0]):
        got = call(qsa, p, good, first)
        others(got)
        s = p.slots(1, np.arange(300))
        assert got[4] == (3, 1) and np.array_equal(got[0][s], p.k[s]) and np.array_equal(got[2][1], p.mass[1])
    # an entry below its place, one past the table, one in the middle of a block: not moved
    for at, t in ((5, 4), (7, 304), (8, 10 ** 9)):
        lists = [x.copy() for x in good]
        lists[1][at] = t
        got = call(qsa, p, lists, [0] * 3)
        others(got)
        assert got[4] == (6, 1)
        assert np.array_equal(got[0][p.slots(1, [at])], p.k[p.slots(1, [at])])
    got = call(qsa, p, good, [0, 2, 0])
    assert got[4] in ((3, 1), (6, 1))
    p.table[1, 0] = p.pages
    got = call(qsa, p, good, [0] * 3)
    others(got)
    assert got[4] == (6, 1)


def test_stream_and_graph(qsa):
    rng = qi.rng_for(65)
    p = Pool(rng, 2, 3000, 16, 512, 2, False)
    lists = [np.sort(rng.permutation(3000)[:1200]), np.arange(1500, 3000)]
    expect = want(p, lists, None)
    same(call(qsa, p, lists, None, stream=torch.cuda.Stream()), expect)
    keep = np.zeros((2, 1500), np.int32)
    for i, x in enumerate(lists):
        keep[i, :len(x)] = x
    k, v, m, st = dev(p.k), dev(p.v), dev(p.mass), qsa.new_status()
    kd, nd, td = dev(keep), dev(np.array([1200, 1500], np.int32)), dev(p.table)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        qsa.qsa_cache_compact(k, v, 512, p.pages, td, p.per, p.per, 16, kd, 1500, nd, 2, 1500, None, m, p.cols, 2, None, None, st)
    g.replay()
    torch.cuda.synchronize()
    assert qsa.qsa_read_status(st) == (0, 0)
    same((k.cpu().numpy().view(np.uint16), v.cpu().numpy().view(np.uint16), m.cpu().numpy()), expect[:3])


def test_serving_loop(qsa, orc):
    """Verify a tree, accept a path, gather its mass, cut the cache back, and go on: the
    attention over the shortened cache and the indexer's scores over the moved
    block keys equal what a cache built from the surviving tokens gives."""
    rng = qi.rng_for(66)
    nq, nkv, hd, page = 8, 2, 128, 16
    c = Cache(rng, [901, 300], [7, 5], nq, nkv, hd, page, "tree")
    scale, row = hd ** -0.5, nq * hd
    d = c.device()
    cols = 912
    st = qsa.new_status()
    out = torch.zeros((c.n_rows, row), dtype=torch.int16, device="cuda")
    lse = torch.zeros((c.n_rows, nq), dtype=torch.float32, device="cuda")
    mass0 = rng.random((2, nkv, cols), dtype=np.float32)
    mass = dev(mass0)
    ws = qsa.new_tree_workspace(2, c.n_rows, nq, nkv, hd)
    tree = (nq, nkv, hd, d["k"], d["v"], c.pages, page, d["table"], c.table_len, c.table_len)
    qsa.qsa_tree_attn(dev(c.q), row, *tree, d["ctx"], d["start"], 2, c.n_rows, d["mask"], c.words, scale, out, row, lse, st, ws)
    for i in range(2):
        want_out, tol, _, _ = ref_tree(c, i, scale)
        r0, m = int(c.row_start[i]), int(c.rows[i])
        got = f64(out.cpu().numpy().view(np.uint16)[r0:r0 + m]).reshape(m, nq, hd)
        assert np.all(np.abs(got - want_out) <= tol)
    # the longest path of each tree is accepted
    paths = []
    for i in range(2):
        sees = c.sees(i)
        leaf = int(np.argmax(sees.sum(1)))
        paths.append(np.nonzero(sees[leaf])[0])
    weight = np.zeros(c.n_rows, np.float32)
    for i, p in enumerate(paths):
        weight[int(c.row_start[i]) + p] = 1.0
    qsa.qsa_attn_mass(dev(c.q), row, nq, nkv, hd, d["k"], c.pages, page, d["table"], c.table_len, c.table_len, d["ctx"],
                      d["start"], 2, c.n_rows, d["mask"], c.words, scale, lse, dev(weight), 0.5, mass, cols, st)
    keep = np.zeros((2, 8), np.int32)
    for i, p in enumerate(paths):
        keep[i, :len(p)] = c.ctx[i] + p
    qsa.qsa_cache_compact(d["k"], d["v"], nkv * hd, c.pages, d["table"], c.table_len, c.table_len, page, dev(keep), 8,
                          dev(np.array([len(p) for p in paths], np.int32)), 2, 8, d["ctx"], mass, cols, nkv, None, None, st)
    length = (c.ctx + np.array([len(p) for p in paths])).astype(np.int32)
    # the indexer's block keys of those contexts
    nb = cols // 4
    raw = qi.raw_keys(rng, 2 * cols).reshape(2, cols, 128)
    qw, kw = qi.norm_weights(rng)
    cos_t, sin_t = qsa.qsa_rope_tables(cols, THETA)
    block_keys = torch.zeros((2 * nb, 128), dtype=torch.int16, device="cuda")
    for i in range(2):
        qsa.qsa_pool_blocks(dev(raw[i]), 128, 0, int(length[i]) // 4, dev(kw), dev(cos_t), dev(sin_t), cols, EPS,
                            block_keys[i * nb:])
    before = block_keys.cpu().numpy().view(np.uint16).copy()
    base = np.array([0, nb], np.int64)
    # cut back to 256 tokens in whole blocks
    budget, first, last = 256, 4, 64
    sel = torch.full((2, budget + 3), -1, dtype=torch.int32, device="cuda")
    n_sel = torch.zeros(2, dtype=torch.int32, device="cuda")
    qsa.qsa_evict_select(mass, cols, nkv, dev(length), 2, cols, budget, first, last, 4, sel, budget + 3, n_sel, st)
    lists = [sel[i, :int(n_sel[i])].cpu().numpy() for i in range(2)]
    m = mass.cpu().numpy()
    for i in range(2):
        assert np.array_equal(lists[i], keep_units(m[i], int(length[i]), budget, first, last, 4))
    pools = d["k"].cpu().numpy().view(np.uint16).copy(), d["v"].cpu().numpy().view(np.uint16).copy()
    qsa.qsa_cache_compact(d["k"], d["v"], nkv * hd, c.pages, d["table"], c.table_len, c.table_len, page, sel, budget + 3, n_sel,
                          2, budget + 3, None, mass, cols, nkv, block_keys, dev(base), st)
    assert qsa.qsa_read_status(st) == (0, 0)
    short = n_sel.cpu().numpy()
    # the next step: one row a sequence, its token written behind the shortened cache
    q1 = qi.normal_bf16(rng, (2, row), 1.5)
    new_kv = qi.normal_bf16(rng, (2, 2, nkv * hd))
    fresh = Cache(rng, short, [1, 1], nq, nkv, hd, page, "chain")
    fresh.q = q1
    for i in range(2):
        at = c.slots(i, [int(short[i])])[0]
        d["k"][at] = dev(new_kv[i, 0])
        d["v"][at] = dev(new_kv[i, 1])
        to = fresh.slots(i, np.arange(short[i] + 1))
        src = c.slots(i, lists[i])
        fresh.k[to] = np.concatenate([pools[0][src], new_kv[i, :1]])
        fresh.v[to] = np.concatenate([pools[1][src], new_kv[i, 1:]])
    out1 = torch.zeros((2, row), dtype=torch.int16, device="cuda")
    qsa.qsa_tree_attn(dev(q1), row, *tree, n_sel, dev(np.array([0, 1, 2], np.int32)), 2, 2, None, 0, scale, out1, row, None, st,
                      ws)
    for i in range(2):
        want_out, tol, _, _ = ref_tree(fresh, i, scale)
        got = f64(out1.cpu().numpy().view(np.uint16)[i:i + 1]).reshape(1, nq, hd)
        assert np.all(np.abs(got - want_out) <= tol)
    # the indexer over the shortened keys: true positions for the rotation, the short length for the blocks
    fq = qi.fused_qk(rng, 2)
    blocks = short // 4
    sc = torch.full((2, nb), -7.0, dtype=torch.float32, device="cuda")
    qsa.qsa_score_rows(dev(fq), 640, dev(length), dev(short), 2, cols, dev(qw), dev(cos_t), dev(sin_t), cols, EPS, block_keys,
                       dev(base), sc, nb, st)
    assert qsa.qsa_read_status(st) == (0, 0)
    got = sc.cpu().numpy()
    for i in range(2):
        kept = before[base[i] + lists[i][:4 * blocks[i]:4] // 4]
        s = np.full((1, nb), -7.0, np.float32)
        rc, _ = orc.score_rows(fq[i:i + 1], 640, length[i:i + 1], 1, cols, qw, cos_t, sin_t, EPS, np.ascontiguousarray(kept), s,
                               nb, visible_len=short[i:i + 1])
        assert rc == 0
        assert np.all(np.abs(got[i, :blocks[i]] - s[0, :blocks[i]]) <= 5e-3 + 1e-3 * np.abs(s[0, :blocks[i]]))
