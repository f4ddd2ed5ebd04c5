"""What a bad sequence leaves of the others."""
import numpy as np
import pytest

import qsa_inputs as qi
from cache_cases import Cache
from test_gpu_mass import call as mass_call
from test_gpu_tree import call as tree_call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("hd", [128, 256])
@pytest.mark.parametrize("n", [3, 40, 500])
def test_starts_that_do_not_ascend_leave_the_good_sequences(qsa, n, hd):
    """A start far above the others, in the middle, makes two sequences bad; one behind them
    owns rows 0..3 of a context that many CTAs share, and another the rows after those."""
    rng = qi.rng_for(80, salt=n + hd)
    ctx, rows = np.full(n, 30), np.zeros(n, int)
    mid = n // 2
    good = [n - 1] if n == 3 else [mid + 1, n - 1]
    for k, i in enumerate(good):
        ctx[i], rows[i] = (9001, 4) if k == 0 else (20, 2)
    c = Cache(rng, ctx, rows, 8, 2, hd, 16, "tree")
    want, wlse, st = tree_call(qsa, c)
    assert st == (0, 0)
    lse = np.where(np.isfinite(wlse), wlse, 0).astype(np.float32)
    old, wmass, st = mass_call(qsa, c, lse)
    assert st == (0, 0)
    c.row_start[mid] = 10 * n + 100  # past n_rows: the sequences on either side contradict themselves
    out, glse, st = tree_call(qsa, c)
    assert st[0] == 3 and st[1] in (mid - 1, mid)
    assert np.array_equal(out, want) and np.array_equal(glse, wlse)
    _, mass, st = mass_call(qsa, c, lse, old=old)
    assert st[0] == 3 and st[1] in (mid - 1, mid)
    assert np.array_equal(mass, wmass)
