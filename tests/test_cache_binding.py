"""The cache operators' Python binding on the host: no GPU, no launch."""
import ctypes
import itertools

import pytest


@pytest.fixture(scope="module")
def qsa():
    import __graft_entry__

    __graft_entry__.build()
    import sparse_attention_token_qsa_gb300 as m

    return m


def test_tree_workspace_refuses_what_the_call_refuses(qsa):
    for bad in ((-1, 1, 16, 2, 256), (1, -1, 16, 2, 256), (1, 1, 0, 2, 256), (1, 1, 16, 0, 256), (1, 1, 15, 2, 256),
                (1, 1, 16, 2, 64)):
        with pytest.raises(ValueError):
            qsa.new_tree_workspace(*bad, device="cpu")
    assert qsa.new_tree_workspace(0, 0, 16, 2, 256, device="cpu").numel() >= 16
    assert qsa.new_tree_workspace(3, 9, 16, 2, 256, device="cpu").numel() == qsa.qsa_tree_workspace_bytes(3, 9, 16, 2, 256)


def test_tree_workspace_grows_with_what_it_says(qsa):
    """Sequences, rows, heads of a group and head_dim; the same heads over fewer KV heads."""
    f = qsa.qsa_tree_workspace_bytes
    for n, rows, group, hd in itertools.product((1, 31, 33, 600), (1, 4, 40, 1000), (1, 4, 8, 130), (128, 256)):
        here = f(n, rows, 8 * group, 8, hd)
        assert here == f(n, rows, group, 1, hd)
        assert here <= f(n + 1, rows, group, 1, hd) and here <= f(n, rows + 1, group, 1, hd)
        assert here <= f(n, rows, group + 1, 1, hd) and here <= f(n, rows, group, 1, 256)
    assert f(4, 4, 16, 2, 128) > f(4, 4, 16, 8, 128)


def test_bounds_that_the_header_names(qsa):
    """Each bound is refused one past it; the same call with nothing to do is no error."""
    lib, P = qsa.library(), ctypes.c_void_p
    A, B = P(0x10000), P(0x20000)  # never read

    def tree(nq=16, nkv=2, n=2, rows=9, pages=100, tl=40):
        return lib.qsa_tree_attn(A, 128 * nq, nq, nkv, 128, A, A, pages, 16, B, tl, tl, B, B, n, rows, None, 0, 0.1, A,
                                 128 * nq, None, B, A, 1 << 60, None)

    def mass(nq=16, nkv=2, n=2, rows=9, pages=100, tl=40):
        return lib.qsa_attn_mass(A, 128 * nq, nq, nkv, 128, A, pages, 16, B, tl, tl, B, B, n, rows, None, 0, 0.1, B, None,
                                 1.0, A, 640, B, None)

    def evict(n=2, nkv=2, tokens=1000):
        return lib.qsa_evict_select(A, (tokens + 3) // 4 * 4, nkv, B, n, tokens, 256, 4, 64, 4, A, 259, B, B, None)

    def compact(n=2, nkv=2, width=512, tl=40):
        return lib.qsa_cache_compact(A, A, width, 100, B, tl, tl, 16, B, 300, B, n, 259, None, A, 640, nkv, None, None, B, None)

    for f in (tree, mass):
        for kw in (dict(n=65536), dict(nq=65536, nkv=65536), dict(rows=1 << 27), dict(pages=1 << 26), dict(tl=1 << 27)):
            assert f(**kw) == 1, kw
        assert f(n=0) == 0
    for f, kws in ((evict, (dict(n=(1 << 20) + 1), dict(nkv=65536), dict(tokens=2 ** 31 - 65536))),
                   (compact, (dict(n=65536), dict(nkv=65536), dict(width=(1 << 24) + 8), dict(tl=1 << 27)))):
        for kw in kws:
            assert f(**kw) == 1, kw
        assert f(n=0) == 0
