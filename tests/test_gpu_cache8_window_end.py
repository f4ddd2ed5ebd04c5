"""Windows as long as the longest tables."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev
from step_cases import Cache8
from test_gpu_cache8 import call, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("nq,nkv,hd", [(2, 2, 128), (4, 1, 256)])
def test_a_window_near_2_31(qsa, nq, nkv, hd):
    """A chunk in a window one short of a table of 2^31 - 512 tokens: token and window together pass 31 bits.  Every row
    sees all of its tokens, as without a window."""
    rng = qi.rng_for(113, salt=hd)
    page = 512
    c = Cache8(rng, [0], [1300], nq, nkv, hd, page, 64, "chain")
    want, wlse, st = call(qsa, c)
    assert st == (0, 0)
    table_len = (2 ** 31 - 257) // page
    table = torch.full((1, table_len), -1, dtype=torch.int32, device="cuda")
    table[0, :c.table_len] = dev(c.table)[0]
    c.table_len, c.window = table_len, table_len * page - 1
    c.device = lambda: dict(Cache8.device(c), table=table)
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    assert np.all(np.isfinite(lse))
    c.window = 0
    check(c, want, wlse)
    check(c, out, lse)
