"""Contexts and rows at the edges of the kernels' tiles of tokens (96 and 64 in tree
attention, 128 in the mass), and rows that count nothing between rows that do."""
import numpy as np
import pytest

import qsa_inputs as qi
from cache_cases import Cache
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
