"""Pages outside the pool in what a plan gives back and takes."""
import numpy as np
import pytest

import qsa_inputs as qi
from step_cases import ref_plan
from test_gpu_plan import case, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


# One CTA, a cluster of them, and more sequences than a CTA's threads
@pytest.mark.parametrize("n", [2, 40, 300, 1500])
@pytest.mark.parametrize("bad", [-1, "pages", 2 ** 31 - 1, -2 ** 31])
def test_a_bad_page_given_back_plans_nothing(qsa, n, bad):
    """It must not come to the stack of free pages, from which another sequence would be given it."""
    rng = qi.rng_for(114, salt=n)
    for s in sorted({0, n // 2, n - 1}):
        c = case(rng, rng.integers(20, 200, n), rng.integers(0, 40, n), 16, slack=4)
        ctx, new, held = c["ctx"], c["new"], c["held"]
        new[s] = 0
        ctx[s] = min(int(ctx[s]), int(held[s] - 1) * 16)  # (it gives back one page at least)
        need = -(-int(ctx[s]) // 16)
        was = int(c["table"][s, need])
        c["table"][s, need] = c["pages"] if bad == "pages" else bad
        for inplace in (False, True):
            got, st, _ = run(qsa, c, inplace=inplace)
            assert st == (6, s)
            assert np.array_equal(got["table"], c["table"]) and np.array_equal(got["held"], held)
            assert got["n_free"] == c["n_free"] and np.array_equal(got["free"][:c["n_free"]], c["free"][:c["n_free"]])
            assert np.all(got["row_start"] == 0) and np.all(got["slot"] == -1)
        c["table"][s, need] = was  # mended: the plan goes on
        check(qsa, c, inplace=True)


def test_a_bad_page_taken_stays_with_its_sequence(qsa):
    """It goes from the stack to the table of the sequence that the status names, and never back."""
    rng = qi.rng_for(115)
    c = case(rng, [40, 100], [9, 13], 16)
    c["free"][c["n_free"] - 1] = c["pages"] + 3  # the first sequence's next page
    got, st, _ = run(qsa, c)
    want, errors = ref_plan(c["ctx"], c["new"], 16, c["table"], c["held"], c["free"], c["n_free"], 22, c["pages"])
    assert not errors and st == (6, 0)
    want["slot"][8] = -1
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    assert got["table"][0, 3] == c["pages"] + 3
    c.update(table=got["table"], held=got["held"], free=got["free"], n_free=got["n_free"],
             ctx=np.array([0, 113], np.int32), new=np.array([0, 15], np.int32))
    got, st, _ = run(qsa, c)
    assert st == (6, 0) and got["n_free"] == c["n_free"] and np.array_equal(got["table"], c["table"])
    assert np.all(got["row_start"] == 0)
