"""Calls whose result depends on the order of a kernel's own copies, stores and waits."""
import numpy as np
import pytest

import qsa_inputs as qi
from cache_cases import Cache
from test_gpu_tree import call as tree_call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("hd", [128, 256])
def test_signs_of_the_scale_and_of_the_query(qsa, hd):
    """A negative scale gives the bits of the negated query under the positive one, and a
    zero scale those of a zero query, over enough units that each CTA fetches Q many times."""
    rng = qi.rng_for(82, salt=hd)
    c = Cache(rng, rng.integers(0, 900, 70), rng.integers(1, 40, 70), 16, 4, hd, 16, "tree")
    plus = c.q.copy()
    for scale, q in ((0.07, plus ^ 0x8000), (1.0, np.zeros_like(plus))):
        c.q = q
        want = tree_call(qsa, c, scale=scale)
        c.q = plus
        for _ in range(5):
            got = tree_call(qsa, c, scale=-scale if scale < 1 else 0.0)
            assert got[2] == (0, 0) and want[2] == (0, 0)
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
