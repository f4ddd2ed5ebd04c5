"""The step operators over very many sequences, single rows beside sequences of many, and calls at once."""
import threading

import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev
from step_cases import Cache8
from test_gpu_cache8 import call as attend, check as check_attend
from test_gpu_plan import case as plan_case, check as check_plan
from test_gpu_write import Write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def test_most_sequences_planned(qsa):
    rng = qi.rng_for(120)
    n = 65535
    check_plan(qsa, plan_case(rng, rng.integers(0, 40, n), rng.integers(0, 2, n), 16, slack=2), inplace=True)


@pytest.mark.parametrize("bits", [8, 16])
def test_many_sequences_written(qsa, bits):
    rng = qi.rng_for(121, salt=bits)
    n = 20000
    c = Write(qsa, rng, rng.integers(0, 17, n), rng.integers(0, 2, n), 1, 1, 128, 16, 16, bits)
    o, got, st = c.run(qsa)
    assert st == (0, 0)
    c.check(o, got)


def test_many_sequences_attended(qsa):
    rng = qi.rng_for(122)
    n = 20000
    c = Cache8(rng, rng.integers(0, 17, n), rng.integers(0, 2, n), 2, 1, 128, 16, 16, "chain")
    out, lse, st = attend(qsa, c)
    assert st == (0, 0)
    check_attend(c, out, lse)


@pytest.mark.parametrize("hd,nq,nkv,mask", [(128, 4, 2, "chain"), (256, 16, 2, "tree")])
def test_wide_sequences_between_single_rows(qsa, hd, nq, nkv, mask):
    """A unit's rows follow the call's mean: here many of them make up the wide sequences."""
    rng = qi.rng_for(123, salt=hd)
    rows = [1] * 150 + [300] + [1] * 60 + [97, 0, 1]
    c = Cache8(rng, rng.integers(0, 300, len(rows)), rows, nq, nkv, hd, 16, 16, mask, n_first=3, window=131)
    out, lse, st = attend(qsa, c)
    assert st == (0, 0)
    check_attend(c, out, lse)


def test_calls_at_once(qsa):
    """Three streams attend one cache, each in a workspace of its own."""
    rng = qi.rng_for(124)
    c = Cache8(rng, [3000, 515, 40], [1, 20, 3], 16, 2, 256, 16, 16, "tree")
    want, wl, st = attend(qsa, c)
    assert st == (0, 0)
    check_attend(c, want, wl)
    d, q, row = c.device(), dev(c.q), c.nq * c.hd
    args = c.args(q, row, d)
    sides = [(torch.cuda.Stream(), torch.zeros((c.n_rows, row), dtype=torch.int16, device="cuda"), qsa.new_status(),
              qsa.new_cache8_workspace(c.n, c.n_rows, c.nq, c.nkv, c.hd)) for _ in range(3)]
    torch.cuda.synchronize()

    def go(s, out, st, ws):
        for _ in range(8):
            qsa.qsa_cache8_attn(*args, c.hd ** -0.5, out, row, None, st, ws, stream=s)

    threads = [threading.Thread(target=go, args=side) for side in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for _, out, st, _ in sides:
        assert qsa.qsa_read_status(st) == (0, 0)
        assert np.array_equal(out.cpu().numpy().view(np.uint16), want)
