"""The waits of the cache's tcgen05 kernels run out: a limit of a few cycles makes the
calls report QSA_ERR_TIMEOUT and return, and the next calls are right again."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import Cache, dev

pytestmark = pytest.mark.gpu


def test_tree_attention_gives_up_and_recovers():
    import sparse_attention_token_qsa_gb300 as qsa

    default = qsa.qsa_wait_limit_cycles()
    for hd in (128, 256):
        c = Cache(qi.rng_for(70, salt=hd), [5000, 40], [5, 9], 8, 2, hd, 16, "tree")
        row = c.nq * hd
        args = c.tree_args(dev(c.q), row)
        ws = qsa.new_tree_workspace(c.n, c.n_rows, c.nq, c.nkv, hd)

        def run():
            out = torch.zeros((c.n_rows, row), dtype=torch.int16, device="cuda")
            st = qsa.new_status()
            qsa.qsa_tree_attn(*args, hd ** -0.5, out, row, None, st, ws)
            return out.cpu().numpy(), qsa.qsa_read_status(st)

        want, st = run()
        assert st == (0, 0)
        try:
            qsa.qsa_set_wait_limit_cycles(1)
            _, st = run()
        finally:
            qsa.qsa_set_wait_limit_cycles(default)
        assert st[0] == 5
        got, st = run()
        assert st == (0, 0) and np.array_equal(got, want)


def test_attention_mass_gives_up_and_recovers():
    import sparse_attention_token_qsa_gb300 as qsa

    default = qsa.qsa_wait_limit_cycles()
    for hd, rows in ((128, 5), (128, 90), (256, 5), (256, 90)):
        c = Cache(qi.rng_for(71, salt=hd + rows), [5000, 40], [rows, 9], 8, 2, hd, 16, "tree")
        args = c.mass_args(dev(c.q), c.nq * hd)
        lse = torch.full((c.n_rows, c.nq), 9.0, dtype=torch.float32, device="cuda")

        def run():
            mass = torch.zeros((2, 2, 5096), dtype=torch.float32, device="cuda")
            st = qsa.new_status()
            qsa.qsa_attn_mass(*args, hd ** -0.5, lse, None, 1.0, mass, 5096, st)
            return mass.cpu().numpy(), qsa.qsa_read_status(st)

        want, st = run()
        assert st == (0, 0)
        try:
            qsa.qsa_set_wait_limit_cycles(1)
            _, st = run()
        finally:
            qsa.qsa_set_wait_limit_cycles(default)
        assert st[0] == 5
        got, st = run()
        assert st == (0, 0) and np.array_equal(got, want)
