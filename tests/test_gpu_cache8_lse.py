"""The lse of qsa_cache8_attn where a row's sum is not finite, and where its reference lies far below the logits."""
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


# Units that CTAs share: a window of a few tokens on both sides of a tile's end.
@pytest.mark.parametrize("hd", [128, 256])
def test_lse_of_shared_units_with_small_scales(qsa, hd):
    """V's scales are 0, so references lie far below the logits, which are 0: lse is the logarithm of the tokens' number,
    to 2^-22 of a logarithm in units of 2, a rounding of its sum with the exponent and one of the product: under 2^-20,
    whatever the reference is."""
    rng = qi.rng_for(111, salt=hd)
    for rows in (1, 6):
        for window in (2, 3, 5, 6, 7, 11, 13, 19, 23, 60, 100):
            c = Cache8(rng, [1280], [rows], 16, 2, hd, 16, 16, "chain", window=window)
            c.vs[:] = 0
            c.q[:] = 0
            out, lse, st = call(qsa, c)
            assert st == (0, 0) and np.all(f64(out) == 0)
            want = np.log(c.sees(0).sum(1).astype(np.float64))[:, None]
            assert np.all(np.abs(lse - want) <= 2.0 ** -20), (rows, window, np.max(np.abs(lse - want)))
