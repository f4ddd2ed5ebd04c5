"""The cases of test_gpu_cache8 with page tables far longer than their contexts, as a server has them: the kernel, which
knows no other bound of the contexts, then takes its widest units."""
import numpy as np
import pytest

import test_gpu_cache8 as base
from step_cases import Cache8
from test_gpu_cache8 import (qsa, test_a_key_far_above_the_others, test_bad_pages_and_scales,  # noqa: F401
                             test_bad_sequences_alone, test_logits_that_grow, test_long_context_beside_short_ones,
                             test_many_sequences, test_nan_stays_with_the_rows_that_see_it, test_queries_of_every_size,
                             test_ragged_batch, test_repeats_its_bits, test_rows_that_see_nothing, test_scales_far_apart,
                             test_scales_of_logits, test_streams_graphs_and_shared_workspace, test_wide_trees_and_chunks,
                             test_windows)

pytestmark = pytest.mark.gpu


class LongTables(Cache8):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        entries = max(self.table_len, 120000 // self.page)
        self.table = np.pad(self.table, ((0, 0), (0, entries - self.table_len)), constant_values=-1)
        self.table_len = entries


@pytest.fixture(autouse=True)
def long_tables(monkeypatch):
    monkeypatch.setattr(base, "Cache8", LongTables)


@pytest.mark.parametrize("nq,nkv,hd,rows", [(32, 8, 128, 330), (24, 2, 256, 170)])
@pytest.mark.parametrize("mask", ["tree", "chain"])
def test_windows_over_many_rows(qsa, nq, nkv, hd, rows, mask):  # noqa: F811
    """Wide units whose rows' windows begin in different tiles, beside a sequence that a window has not reached."""
    for n_first, window in ((0, 131), (5, 64)):
        c = Cache8(base.qi.rng_for(130, salt=rows + window), [500, 0], [rows, rows // 2], nq, nkv, hd, 16, 16, mask,
                   n_first=n_first, window=window)
        out, lse, st = base.call(qsa, c)
        assert st == (0, 0)
        base.check(c, out, lse)


def test_sequences_over_the_same_rows(qsa):  # noqa: F811
    """Starts 0, 300, 0, 300, ...: every other sequence is bad, the good ones have the same rows and the same cache, and
    more units are split between CTAs than as many rows of sequences apart would make."""
    c = Cache8(base.qi.rng_for(131), [1000] * 5, [300, 0, 0, 0, 0], 8, 1, 128, 16, 16, "chain")
    c.table[:] = c.table[0]
    c.row_start = np.array([0, 300, 0, 300, 0, 300], np.int32)
    out, lse, st = base.call(qsa, c)
    assert st[0] == 3 and st[1] in (1, 3)
    base.check(c, out, lse, seqs=[0])
