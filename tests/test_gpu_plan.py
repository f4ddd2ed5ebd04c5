"""qsa_page_plan against the plain form: whole numbers, equal."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import dev
from step_cases import ref_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


def case(rng, ctx, new, page, slack=0, spare=None, cols_pad=0):
    """A pool whose pages are in tables or on the stack; sequences hold their context's pages and up to `slack` more."""
    ctx, new = np.asarray(ctx, np.int32), np.asarray(new, np.int32)
    n = len(ctx)
    held = (-(-ctx // page) + (rng.integers(0, slack + 1, n) if slack else 0)).astype(np.int32)
    need = -(-(ctx + new) // page)
    take = int(np.maximum(0, need - held).sum())
    pages = int(held.sum()) + (take + 3 if spare is None else spare)
    pages = max(1, pages)
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((n, max(1, int(max(held.max(), need.max())))), -7, np.int32)
    at = 0
    for s in range(n):
        table[s, :held[s]] = order[at:at + held[s]]
        at += int(held[s])
    free = np.full(pages, -9, np.int32)
    free[:pages - at] = order[at:]
    return dict(ctx=ctx, new=new, page=page, table=table, held=held, free=free, n_free=pages - at, pages=pages, pad=cols_pad)


def run(qsa, c, max_rows=None, inplace=False, optional=True, stream=None):
    n, cols = c["table"].shape
    pad = np.full((n, cols + c["pad"]), -11, np.int32)
    pad[:, :cols] = c["table"]
    max_rows = int(c["new"].sum()) if max_rows is None else max_rows
    t, held, free, nf = dev(pad), dev(c["held"]), dev(c["free"]), dev(np.array([c["n_free"]], np.int32))
    full = lambda k: torch.full((k,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    ho, nfo = (held, nf) if inplace else (full(n), full(1))
    start, slot, pos, seq = full(n + 2), full(max_rows + 1), full(max_rows + 1), full(max_rows + 1)
    st = qsa.new_status()
    ctx, new = dev(c["ctx"]), dev(c["new"])
    torch.cuda.synchronize()
    qsa.qsa_page_plan(ctx, new, n, c["page"], c["pages"], t, cols, cols + c["pad"], held, ho, free, nf, nfo, max_rows, start,
                      slot, pos if optional else None, seq if optional else None, st, stream=stream)
    torch.cuda.synchronize()
    back = dict(table=t, held=ho, free=free, n_free=nfo, row_start=start, slot=slot, pos=pos, row_seq=seq)
    got = {k: x.cpu().numpy() for k, x in back.items()}
    assert np.all(got["table"][:, cols:] == -11) and got["row_start"][-1] == -77
    got["table"], got["row_start"], got["n_free"] = got["table"][:, :cols], got["row_start"][:-1], int(got["n_free"][0])
    for k in ("slot", "pos", "row_seq"):
        assert got[k][-1] == -77, k
        got[k] = got[k][:-1]
    return got, qsa.qsa_read_status(st), max_rows


def check(qsa, c, **kw):
    got, st, max_rows = run(qsa, c, **kw)
    want, errors = ref_plan(c["ctx"], c["new"], c["page"], c["table"], c["held"], c["free"], c["n_free"], max_rows, c["pages"])
    skip = () if kw.get("optional", True) else ("pos", "row_seq")
    for k in want:
        if k not in skip:
            assert np.array_equal(got[k], want[k]), k
    if errors:
        assert st in errors
    else:
        assert st == (0, 0)
    return got


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("n", [1, 3, 31, 32, 33, 250, 257])
def test_ragged(qsa, n, page):
    rng = qi.rng_for(40, salt=n * 100 + page)
    c = case(rng, rng.integers(0, 200, n), rng.integers(0, 40, n), page, slack=int(rng.integers(0, 6)), cols_pad=3)
    check(qsa, c)
    check(qsa, c, inplace=True)
    check(qsa, c, optional=False)
    check(qsa, c, max_rows=int(c["new"].sum()) + 70)


def test_lengths_at_the_pages_edges(qsa):
    rng = qi.rng_for(41)
    ctx = [0, 0, 0, 1, 15, 15, 16, 16, 17, 32, 31, 0]
    new = [0, 1, 16, 0, 1, 2, 0, 1, 15, 17, 0, 33]
    for slack in (0, 2):
        check(qsa, case(rng, ctx, new, 16, slack=slack), inplace=True)


def test_no_rows_at_all(qsa):
    rng = qi.rng_for(42)
    got = check(qsa, case(rng, [3, 0, 40], [0, 0, 0], 16), max_rows=0)
    assert np.all(got["row_start"] == 0)
    check(qsa, case(rng, [3, 0, 40], [0, 0, 0], 16), max_rows=5)


@pytest.mark.parametrize("n", [1, 1023, 1024, 1025, 3000])
def test_many_sequences_and_rows(qsa, n):
    """More than a CTA's threads, sequences without rows between ones with many, pages given back and taken again."""
    rng = qi.rng_for(43, salt=n)
    new = rng.integers(0, 3, n)
    new[rng.integers(0, n, 3)] = [9000, 700, 65]
    c = case(rng, rng.integers(0, 400, n), new, 16, slack=9, spare=None)
    check(qsa, c, inplace=True)
    check(qsa, c, max_rows=int(new.sum()) + 1000)


def test_given_back_pages_serve_the_call(qsa):
    """The stack is empty before: what is taken is what others gave back, in the documented order."""
    rng = qi.rng_for(44)
    c = case(rng, [100, 5, 64], [0, 60, 1], 16, spare=0)
    c["held"] = np.array([7, 1, 4], np.int32)
    c["ctx"] = np.array([17, 5, 64], np.int32)  # the first gives back five, the others need five
    c["new"] = np.array([0, 59, 1], np.int32)
    got = check(qsa, c, inplace=True)
    assert got["n_free"] == 1


@pytest.mark.parametrize("n", [40, 400])
def test_too_few_pages_rows_or_room(qsa, n):
    """Nothing is planned, and the state stays as it was."""
    rng = qi.rng_for(45, salt=n)
    c = case(rng, rng.integers(0, 200, n), rng.integers(1, 40, n), 16, slack=2)
    c["n_free"] -= 5
    check(qsa, c)  # enough all the same: the pages that others give back serve
    need = -(-(c["ctx"] + c["new"]) // 16)
    c["n_free"] = int((need - c["held"]).sum()) - 1
    for inplace in (False, True):
        got = check(qsa, c, inplace=inplace)
        assert np.all(got["row_start"] == 0) and np.array_equal(got["held"], c["held"]) and np.all(got["slot"] == -1)
    c = case(rng, rng.integers(0, 200, n), rng.integers(1, 40, n), 16)
    got = check(qsa, c, max_rows=int(c["new"].sum()) - 1)
    assert np.all(got["row_start"] == 0)
    c["n_free"] = -1
    check(qsa, c)
    c = case(rng, [40] * n, [0] * n, 16, slack=3)
    c["n_free"] = c["pages"]
    check(qsa, c)


@pytest.mark.parametrize("n", [9, 300])
def test_bad_sequences_alone(qsa, n):
    rng = qi.rng_for(46, salt=n)
    good = case(rng, rng.integers(0, 200, n), rng.integers(0, 40, n), 16, slack=2)
    cols = good["table"].shape[1]
    for which, value in (("ctx", -1), ("new", -3), ("held", -1), ("held", cols + 1), ("ctx", cols * 16 + 1), ("new", 2 ** 31 - 1),
                         ("ctx", 2 ** 31 - 1)):
        for s in (0, n // 2, n - 1):
            c = {k: (x.copy() if isinstance(x, np.ndarray) else x) for k, x in good.items()}
            c[which][s] = value
            got, st, _ = run(qsa, c, max_rows=int(good["new"].sum()))
            want, errors = ref_plan(c["ctx"], c["new"], 16, c["table"], c["held"], c["free"], c["n_free"],
                                    int(good["new"].sum()), c["pages"])
            assert st == (3, s) and errors == [(3, s)]
            for k in want:
                assert np.array_equal(got[k], want[k]), (which, value, s, k)


def test_pages_outside_the_pool(qsa):
    rng = qi.rng_for(47)
    for bad in (-1, 10 ** 6):
        c = case(rng, [40, 100], [9, 3], 16)
        c["free"][c["n_free"] - 1] = bad  # the first sequence's next page
        got, st, _ = run(qsa, c)
        assert st == (6, 0)
        assert list(got["slot"][:8] >= 0) == [True] * 8 and got["slot"][8] == -1 and np.all(got["slot"][9:] >= 0)
        c = case(rng, [40, 100], [9, 3], 16)
        c["table"][1, 6] = bad
        got, st, _ = run(qsa, c)
        assert st == (6, 1) and np.all(got["slot"][:9] >= 0) and np.all(got["slot"][9:] == -1)


def test_captured_steps_in_place(qsa):
    """A graph of one plan, replayed while the lengths grow by the rows: the same as the plain steps."""
    rng = qi.rng_for(48)
    n, page = 37, 16
    c = case(rng, rng.integers(0, 60, n), rng.integers(1, 4, n), page, spare=400)
    cols = 40
    table = np.full((n, cols), -7, np.int32)
    table[:, :c["table"].shape[1]] = c["table"]
    c["table"] = table
    rows = int(c["new"].sum())
    ctx, new, t, held, free, nf = (dev(x) for x in (c["ctx"], c["new"], table, c["held"], c["free"],
                                                   np.array([c["n_free"]], np.int32)))
    start, slot, pos, seq = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (n + 1, rows, rows, rows))
    st = qsa.new_status()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        qsa.qsa_page_plan(ctx, new, n, page, c["pages"], t, cols, cols, held, held, free, nf, nf, rows, start, slot, pos, seq, st)
        ctx.add_(new)
    want = dict(table=table, held=c["held"], free=c["free"], n_free=c["n_free"])
    at = c["ctx"].copy()
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        want, errors = ref_plan(at, c["new"], page, want["table"], want["held"], want["free"], want["n_free"], rows, c["pages"])
        at = at + c["new"]
        assert not errors
        for k, x in (("table", t), ("held", held), ("slot", slot), ("pos", pos), ("row_seq", seq), ("row_start", start)):
            assert np.array_equal(x.cpu().numpy(), want[k]), k
        assert int(nf.item()) == want["n_free"]
        assert np.array_equal(free.cpu().numpy()[:want["n_free"]], want["free"][:want["n_free"]])
    assert qsa.qsa_read_status(st) == (0, 0)
