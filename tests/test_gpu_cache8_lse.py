"""The lse of qsa_cache8_attn where a row's sum is not finite, in units that one CTA holds whole."""
import numpy as np
import pytest

import qsa_inputs as qi
from cache_cases import f64
from step_cases import Cache8
from test_gpu_cache8 import call, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


# Tables of one tile, which leave no unit to share; 40 rows of a KV head a sequence, in units of 8, 16, 32 and 64.
@pytest.mark.parametrize("n", [4, 16, 40, 60])
@pytest.mark.parametrize("hd", [128, 256])
def test_nan_in_whole_units(qsa, hd, n):
    rng = qi.rng_for(110, salt=hd + n)
    c = Cache8(rng, rng.integers(0, 110, n), [10] * n, 8, 2, hd, 16, 16, "chain")
    assert c.table_len * 16 <= 128
    some = (0, n // 2, n - 1)
    out, lse, st = call(qsa, c)
    assert st == (0, 0)
    check(c, out, lse, seqs=some)
    # a K row of a drafted token, which the rows from its own on see; a value of a query head
    c.k[c.slots(0, int(c.ctx[0]) + 4), 1, 9] = 0x7F
    hit = np.zeros(lse.shape, bool)
    hit[4:10, 4:] = True
    for value in (np.nan, np.inf, -np.inf):
        c.q[int(c.row_start[n - 1]) + 3, 5 * hd + 7] = qi.to_bf16_bits(np.array([value], np.float32))[0]
        hit[int(c.row_start[n - 1]) + 3, 5] = True
        got, glse, st = call(qsa, c)
        assert st == (0, 0)
        assert np.all(np.isnan(glse[hit])) and np.array_equal(glse[~hit], lse[~hit])
        nan = np.repeat(hit, hd, axis=1)
        assert np.all(np.isnan(f64(got)[nan])) and np.array_equal(got[~nan], out[~nan])
