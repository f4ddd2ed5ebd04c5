"""qsa_qkv_write beside a table entry outside the pool, and captured."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev
from test_gpu_write import SENT, Write

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("nq,nkv,hd,page,unit", [(4, 2, 128, 16, 16), (16, 2, 256, 32, 16), (8, 1, 128, 64, 64)])
def test_a_bad_entry_loses_its_own_tokens_alone(qsa, nq, nkv, hd, page, unit, bits):
    """Queries, the other pages' K, V and scales and the other sequences are as they would be with a good entry; the bad
    page's tokens go nowhere."""
    rng = qi.rng_for(116, salt=hd + page)
    for entry in (0, 1, 2):
        c = Write(qsa, rng, [20, page // 2 - 1, 33], [5, 2 * page + 3, 9], nq, nkv, hd, page, unit, bits)
        o, clean, st = c.run(qsa)
        assert st == (0, 0)
        c.check(o, clean)
        was = int(c.table[1, entry])
        for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
            c.table[1, entry] = bad
            o2, got, st = c.run(qsa)
            assert st == (6, 1) and np.array_equal(o2, o)
            lost = np.zeros(c.pages * page, bool)
            lost[was * page:(was + 1) * page] = True
            for which in (0, 1):
                before, after = (c.k, c.v)[which], got[which]
                assert np.array_equal(after[lost], before[lost]) and np.array_equal(after[~lost], clean[which][~lost])
                if bits == 8:
                    gone = lost[::unit]
                    scales = (c.ks, c.vs)[which]
                    assert np.array_equal(got[2 + which][gone], scales[gone])
                    assert np.array_equal(got[2 + which][~gone], clean[2 + which][~gone])


@pytest.mark.parametrize("bits", [8, 16])
def test_captured_and_replayed(qsa, bits):
    """A captured write, replayed over fresh pools and other inputs in the same buffers."""
    rng = qi.rng_for(117, salt=bits)
    nq, nkv, hd, n = 8, 2, 128, 3
    cases = [Write(qsa, qi.rng_for(118, salt=i), [5, 30, 64], [40, 3, 1], nq, nkv, hd, 16, 16, bits) for i in range(3)]
    want = [c.run(qsa) for c in cases]
    first, d = cases[0], nq * hd
    x = torch.zeros(first.x.shape, dtype=torch.int16, device="cuda")
    opt = lambda a: None if a is None else torch.zeros_like(dev(a))  # noqa: E731
    bufs = [opt(a) for a in (first.k, first.v, first.ks, first.vs, first.qw, first.kw, first.table)]
    out = torch.full((first.n_rows, d), SENT, dtype=torch.int16, device="cuda")
    st, cos, sin, ctx, start = qsa.new_status(), dev(first.cos), dev(first.sin), dev(first.ctx), dev(first.row_start)
    stride = x.shape[1]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        qsa.qsa_qkv_write(x[:, :d], stride, nq, x[:, d:], stride, x[:, d + nkv * hd:], stride, nkv, hd, bufs[4], bufs[5], first.eps,
                          cos, sin, first.table_rows, None, ctx, start, n, first.n_rows, *bufs[:4], 16, first.pages, 16, bufs[6],
                          first.table_len, first.table_len, out, d, st)
    for i in rng.permutation(6) % 3:
        c = cases[i]
        x.copy_(dev(c.x))
        for b, a in zip(bufs, (c.k, c.v, c.ks, c.vs, c.qw, c.kw, c.table)):
            if b is not None:
                b.copy_(dev(a))
        out.fill_(SENT)
        graph.replay()
        torch.cuda.synchronize()
        o, pools, _ = want[i]
        assert np.array_equal(out.cpu().numpy().view(np.uint16), o)
        for b, p in zip(bufs[:4], pools):
            assert b is None or np.array_equal(b.cpu().numpy().view(p.dtype), p)
    assert qsa.qsa_read_status(st) == (0, 0)
