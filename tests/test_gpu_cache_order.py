"""Calls whose result depends on the order of a kernel's own copies, stores and waits."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev
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


def test_calls_in_turn_on_one_workspace(qsa):
    """Calls of other plans, other parts and other row counts follow each other on one
    workspace without a wait in between: each joins its own parts."""
    cs = []
    for i, (n, rows, hd) in enumerate(((1, 1, 256), (33, 3, 128), (2, 60, 256), (5, 20, 128), (600, 1, 128), (1, 128, 128))):
        rng = qi.rng_for(83, salt=i)
        ctx = rng.integers(0, 40 if n > 33 else 6000 // n, n)
        ctx[n // 2] = 6000
        cs.append(Cache(rng, ctx, np.full(n, rows), 8, 2, hd, 16, "tree"))
    want = [tree_call(qsa, c)[:2] for c in cs]
    ws = max((qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd) for c in cs), key=lambda w: w.numel())
    calls = []
    for c in cs:
        row = c.nq * c.hd
        calls.append((c.tree_args(dev(c.q), row), row, c.hd ** -0.5,
                      torch.zeros((4, c.n_rows, row), dtype=torch.int16, device="cuda"),
                      torch.zeros((4, c.n_rows, c.nq), dtype=torch.float32, device="cuda")))
    st = qsa.new_status()
    torch.cuda.synchronize()
    for k in range(4):
        for args, row, scale, out, lse in calls if k % 2 else calls[::-1]:
            qsa.qsa_tree_attn(*args, scale, out[k], row, lse[k], st, ws)
    torch.cuda.synchronize()
    assert qsa.qsa_read_status(st) == (0, 0)
    for (_, _, _, out, lse), (o, l) in zip(calls, want):
        for k in range(4):
            assert np.array_equal(out[k].cpu().numpy().view(np.uint16), o) and np.array_equal(lse[k].cpu().numpy(), l)
