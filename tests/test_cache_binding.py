"""The cache operators' Python binding on the host: no GPU, no launch."""
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
