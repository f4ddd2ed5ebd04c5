"""Contexts and rows at the edges of the kernels' tiles of tokens (96 and 64 in tree
attention, 128 in the mass), and rows that count nothing between rows that do."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev
from test_gpu_mass import call as mass_call
from test_gpu_mass import check as mass_check
from test_gpu_mass import lse_of
from test_gpu_tree import call as tree_call
from test_gpu_tree import check as tree_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
@pytest.mark.parametrize("rows", [1, 5, 33])
@pytest.mark.parametrize("hd", [128, 256])
def test_edges_of_tiles(qsa, hd, rows, mask):
    """The context, or the context and its drafted tokens, end one before, at and one past
    each of the first two tiles."""
    ends = [t * k + d for t in (64, 96, 128) for k in (1, 2) for d in (-1, 0, 1)]
    ctx = sorted(set(ends + [e - rows for e in ends]))
    c = Cache(qi.rng_for(84, salt=hd + rows), ctx, [rows] * len(ctx), 4, 2, hd, 16, mask)
    out, lse, st = tree_call(qsa, c)
    assert st == (0, 0)
    tree_check(c, out, lse)
    given = lse_of(c, hd ** -0.5)
    old, got, st = mass_call(qsa, c, given, carry=0.5)
    assert st == (0, 0)
    mass_check(c, given, None, 0.5, old, got)


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("carry", [0.0, 0.5, 1.0])
def test_a_sequence_whose_rows_all_count_nothing(qsa, hd, carry):
    """Every draft of the middle sequences is rejected: their mass decays, and their drafted
    tokens' is zero."""
    c = Cache(qi.rng_for(85, salt=hd), [300, 1000, 129, 40], [9, 20, 1, 5], 8, 2, hd, 16, "tree")
    weight = np.ones(c.n_rows, np.float32)
    weight[9:30] = 0.0
    given = lse_of(c, hd ** -0.5)
    old, got, st = mass_call(qsa, c, given, weight, carry)
    assert st == (0, 0)
    mass_check(c, given, weight, carry, old, got)
    for i, m in ((1, 20), (2, 1)):
        x = int(c.ctx[i])
        assert np.array_equal(got[i][:, :x], np.float32(carry) * old[i][:, :x]) and np.all(got[i][:, x:x + m] == 0)


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("nq,nkv,ctx,rows", [(6, 2, [140, 0], [300, 9]), (130, 1, [200, 9], [4, 3]), (300, 1, [200, 9], [3, 3]),
                                             (16, 2, [90, 700, 3], [200, 150, 70])])
def test_rows_without_weight_among_several_turns(qsa, hd, nq, nkv, ctx, rows):
    """More pairs than a turn holds, about a third of the rows of weight zero, runs of more
    than 32 of them among those, also at the beginning and at the end."""
    rng = qi.rng_for(86, salt=hd + nq)
    c = Cache(rng, ctx, rows, nq, nkv, hd, 16, "tree")
    weight = rng.choice([0.0, 1.0, 0.5, -2.0], size=c.n_rows, p=[0.34, 0.33, 0.23, 0.1]).astype(np.float32)
    for i in range(c.n):
        r0, m = int(c.row_start[i]), int(c.rows[i])
        if m > 60:
            weight[r0:r0 + 5] = 0.0
            weight[r0 + m // 2 - 20:r0 + m // 2 + 20] = 0.0
            weight[r0 + m - 3:r0 + m] = 0.0
        else:
            weight[r0 + m // 2] = 0.0
    given = lse_of(c, hd ** -0.5)
    old, got, st = mass_call(qsa, c, given, weight, 0.5)
    assert st == (0, 0)
    mass_check(c, given, weight, 0.5, old, got)
    again = mass_call(qsa, c, given, weight, 0.5, old=old)[1]
    assert np.array_equal(got, again)


@pytest.mark.parametrize("hd", [128, 256])
def test_pages_past_32_bits(qsa, hd):
    """The sequences' pages at the far end of pools of over 2^31 values (2^32 bytes): the bits
    of the same pages in a small pool."""
    rng = qi.rng_for(87, salt=hd)
    c = Cache(rng, [700, 90], [5, 40], 8, 2, hd, 16, "tree")
    width, row = 2 * hd, 8 * hd
    out, lse, st = tree_call(qsa, c)
    old, mass, st2 = mass_call(qsa, c, np.where(np.isfinite(lse), lse, 0).astype(np.float32))
    assert st == (0, 0) and st2 == (0, 0)
    far = (1 << 31) // (16 * width) + 11  # pages before ours
    pages = far + c.pages
    pools = []
    for small in (c.k, c.v):
        big = torch.empty((pages * 16, width), dtype=torch.int16, device="cuda")
        big[far * 16:] = dev(small)
        pools.append(big)
    table = np.where(c.table >= 0, c.table + far, -1).astype(np.int32)
    d, td, st = c.device(), dev(table), qsa.new_status()
    o = torch.full((c.n_rows, row), 0x7FAB, dtype=torch.int16, device="cuda")
    l = torch.full((c.n_rows, 8), 123.0, dtype=torch.float32, device="cuda")
    qsa.qsa_tree_attn(dev(c.q), row, 8, 2, hd, *pools, pages, 16, td, c.table_len, c.table_len, d["ctx"], d["start"], c.n,
                      c.n_rows, d["mask"], c.words, hd ** -0.5, o, row, l, st,
                      qsa.new_tree_workspace(c.n, c.n_rows, 8, 2, hd))
    assert np.array_equal(o.cpu().numpy().view(np.uint16), out) and np.array_equal(l.cpu().numpy(), lse)
    m = dev(old)
    qsa.qsa_attn_mass(dev(c.q), row, 8, 2, hd, pools[0], pages, 16, td, c.table_len, c.table_len, d["ctx"], d["start"], c.n,
                      c.n_rows, d["mask"], c.words, hd ** -0.5, l, None, 1.0, m, old.shape[2], st)
    assert np.array_equal(m.cpu().numpy(), mass)
    keep = np.sort(rng.permutation(700)[:300]).astype(np.int32)[None].repeat(2, 0)
    keep[1, :50] = np.sort(rng.permutation(90)[:50])
    qsa.qsa_cache_compact(*pools, width, pages, td, c.table_len, c.table_len, 16, dev(keep), 300,
                          dev(np.array([300, 50], np.int32)), 2, 300, None, None, 0, 0, None, None, st)
    assert qsa.qsa_read_status(st) == (0, 0)
    for pool, small in zip(pools, (c.k, c.v)):
        want = small.copy()
        for i, n in enumerate((300, 50)):
            want[c.slots(i, np.arange(n))] = small[c.slots(i, keep[i, :n])]
        assert np.array_equal(pool[far * 16:].cpu().numpy().view(np.uint16), want)
