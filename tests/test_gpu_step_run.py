"""Steps of a serving loop: pages planned, heads prepared and written, the cache attended,
one after another and as one captured graph."""
import numpy as np
import pytest
import torch

import qsa_inputs as qi
from cache_cases import BF, Cache, dev, f64, ref_tree
from step_cases import E4M3, Cache8, ref_attend, ref_heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import sparse_attention_token_qsa_gb300 as m

    return m


class Loop:
    """A pool, its free pages and n sequences that start empty."""

    def __init__(self, qsa, rng, n, nq, nkv, hd, page, unit, bits, pages, cols, max_rows, n_first=0, window=0, max_pos=512):
        self.qsa, self.rng, self.n, self.nq, self.nkv, self.hd, self.page, self.unit, self.bits = qsa, rng, n, nq, nkv, hd, page, unit, bits
        self.pages, self.cols, self.max_rows, self.n_first, self.window = pages, cols, max_rows, n_first, window
        tokens = pages * page
        kind = torch.uint8 if bits == 8 else torch.int16
        self.k, self.v = (torch.full((tokens, nkv, hd), 0x7F, dtype=kind, device="cuda") for _ in range(2))
        self.ks, self.vs = ((torch.full((tokens // unit, nkv), float("nan"), device="cuda") for _ in range(2))
                            if bits == 8 else (None, None))
        i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
        self.table, self.held = i32(np.full((n, cols), -1)), i32([0] * n)
        self.free, self.n_free = i32(rng.permutation(pages)), i32([pages])
        self.start, self.slot, self.pos, self.seq = (i32([0] * k) for k in (n + 1, max_rows, max_rows, max_rows))
        self.ctx = i32([0] * n)
        self.qw, self.kw = (qi.normal_bf16(rng, (hd,), 0.1) for _ in range(2))
        self.cos, self.sin = qsa.qsa_rope_tables(max_pos, 10000.0)
        self.cd, self.sd, self.qwd, self.kwd = dev(self.cos), dev(self.sin), dev(self.qw), dev(self.kw)
        self.st = qsa.new_status()
        self.width = (nq + 2 * nkv) * hd
        self.x = torch.zeros((max_rows, self.width), dtype=torch.int16, device="cuda")
        self.q, self.out = (torch.zeros((max_rows, nq * hd), dtype=torch.int16, device="cuda") for _ in range(2))
        self.lse = torch.zeros((max_rows, nq), device="cuda")
        self.new = i32([0] * n)
        self.ws = (qsa.new_cache8_workspace if bits == 8 else qsa.new_tree_workspace)(n, max_rows, nq, nkv, hd)

    def launch(self):
        q, d, nkvd = self.qsa, self.nq * self.hd, self.nkv * self.hd
        x = self.x
        q.qsa_page_plan(self.ctx, self.new, self.n, self.page, self.pages, self.table, self.cols, self.cols, self.held, self.held,
                        self.free, self.n_free, self.n_free, self.max_rows, self.start, self.slot, self.pos, self.seq, self.st)
        q.qsa_qkv_write(x, self.width, self.nq, x[:, d:], self.width, x[:, d + nkvd:], self.width, self.nkv, self.hd, self.qwd,
                        self.kwd, 1e-6, self.cd, self.sd, self.cos.shape[0], self.pos, self.ctx, self.start, self.n, self.max_rows,
                        self.k, self.v, self.ks, self.vs, self.unit, self.pages, self.page, self.table, self.cols, self.cols,
                        self.q, d, self.st)
        head = (self.q, d, self.nq, self.nkv, self.hd, self.k, self.v)
        tail = (self.pages, self.page, self.table, self.cols, self.cols, self.ctx, self.start, self.n, self.max_rows, None, 0)
        if self.bits == 8:
            q.qsa_cache8_attn(*head, self.ks, self.vs, self.unit, *tail, self.n_first, self.window, self.hd ** -0.5, self.out, d,
                              self.lse, self.st, self.ws)
        else:
            q.qsa_tree_attn(*head, *tail, self.hd ** -0.5, self.out, d, self.lse, self.st, self.ws)

    def case(self):
        """The cache as it lies on the GPU, for the plain forms."""
        c = (Cache8 if self.bits == 8 else Cache).__new__(Cache8 if self.bits == 8 else Cache)
        c.ctx, c.rows = self.ctx.cpu().numpy(), self.new.cpu().numpy()
        c.nq, c.nkv, c.hd, c.page, c.unit, c.n, c.group = self.nq, self.nkv, self.hd, self.page, self.unit, self.n, self.nq // self.nkv
        c.n_first, c.window, c.mask, c.words = self.n_first, self.window, None, 0
        c.table, c.row_start = self.table.cpu().numpy(), self.start.cpu().numpy()
        c.q = self.q.cpu().numpy().view(np.uint16)
        c.k, c.v = self.k.cpu().numpy(), self.v.cpu().numpy()
        if self.bits == 8:
            c.ks, c.vs = self.ks.cpu().numpy(), self.vs.cpu().numpy()
        else:
            c.k, c.v = (a.view(np.uint16).reshape(a.shape[0], -1) for a in (c.k, c.v))
        return c

    def step(self, new, history):
        """One step of `new` rows a sequence; checks what it leaves, and adds the tokens' true K and V to `history`."""
        total = int(sum(new))
        x = qi.normal_bf16(self.rng, (self.max_rows, self.width), 2.0)
        self.x.copy_(dev(x))
        self.new.copy_(dev(np.asarray(new, np.int32)))
        self.launch()
        torch.cuda.synchronize()
        assert self.qsa.qsa_read_status(self.st) == (0, 0)
        c = self.case()
        assert np.array_equal(c.row_start, np.concatenate([[0], np.cumsum(new)]))
        pos, slot = self.pos.cpu().numpy(), self.slot.cpu().numpy()
        xs = f64(x)
        d, nkvd = self.nq * self.hd, self.nkv * self.hd
        for i in range(self.n):
            r = np.arange(c.row_start[i], c.row_start[i + 1])
            at = c.ctx[i] + np.arange(len(r))
            assert np.array_equal(pos[r], at) and np.array_equal(slot[r], c.slots(i, at) if len(r) else at)
            q, tol = ref_heads(xs[r, :d].reshape(len(r), self.nq, self.hd), f64(self.qw), 1e-6, f64(self.cos[at]), f64(self.sin[at]))
            assert np.all(np.abs(f64(c.q[r]).reshape(q.shape) - q) <= tol + BF * np.abs(q) + 1e-30)
            k, _ = ref_heads(xs[r, d:d + nkvd].reshape(len(r), self.nkv, self.hd), f64(self.kw), 1e-6, f64(self.cos[at]), f64(self.sin[at]))
            v = xs[r, d + nkvd:].reshape(len(r), self.nkv, self.hd)
            for h, new_rows in zip(history[i], (k, v)):
                del h[c.ctx[i]:]
                h.extend(new_rows)
            kv = int(c.ctx[i]) + len(r)
            if kv == 0:
                continue
            where = c.slots(i, np.arange(kv))
            for pool, scale, true in ((c.k, getattr(c, "ks", None), history[i][0]), (c.v, getattr(c, "vs", None), history[i][1])):
                true = np.array(true)
                if self.bits == 16:
                    assert np.all(np.abs(f64(pool[where]).reshape(true.shape) - true) <= BF * np.abs(true) + 1e-5 * np.abs(true).max())
                else:
                    # a block's scale may have grown since a token was written: below 2^-6 of it, a value
                    # was rounded again, by 2^-10 of the scale of that day, and scales double at least
                    s = scale[where // self.unit].astype(np.float64)[:, :, None]
                    assert np.all(np.abs(E4M3[pool[where]] * s - true) <= 1.001 * 2.0 ** -4 * np.abs(true) + 2 * 2.0 ** -10 * s + 1e-30)
        out, lse = self.out.cpu().numpy().view(np.uint16), self.lse.cpu().numpy()
        for i in range(self.n):
            m, r0 = int(c.rows[i]), int(c.row_start[i])
            want, tol, wl, ltol = (ref_attend if self.bits == 8 else ref_tree)(c, i, self.hd ** -0.5)
            got = f64(out[r0:r0 + m]).reshape(want.shape)
            assert np.all(np.abs(got - want) <= tol), f"sequence {i}"
            assert np.all(np.abs(lse[r0:r0 + m] - wl) <= ltol)
        return total


@pytest.mark.parametrize("bits,nq,nkv,hd,page,unit,n_first,window", [(8, 8, 2, 128, 32, 16, 0, 0), (8, 16, 2, 256, 16, 16, 3, 40),
                                                                      (16, 8, 2, 128, 7, 16, 0, 0)])
def test_a_loop_of_steps(qsa, bits, nq, nkv, hd, page, unit, n_first, window):
    """Prompts, single tokens, drafted chains of which some are taken back, a sequence that ends and one that begins in
    its pages; pages that nobody holds are all free at the end."""
    rng = qi.rng_for(90, salt=bits + hd)
    loop = Loop(qsa, rng, 4, nq, nkv, hd, page, unit, bits, pages=-(-700 // page), cols=-(-300 // page), max_rows=160,
                n_first=n_first, window=window)
    history = [([], []) for _ in range(4)]
    ctx = np.zeros(4, np.int32)

    def step(new, then):
        nonlocal ctx
        loop.step(new, history)
        ctx = np.asarray(then, np.int32)
        loop.ctx.copy_(dev(ctx))

    step([70, 1, 33, 0], [70, 1, 33, 0])
    for _ in range(3):
        step([1, 1, 1, 0], ctx + [1, 1, 1, 0])
    step([5, 4, 1, 0], ctx + [2, 4, 1, 0])      # the first keeps two of its five drafted tokens
    step([1, 6, 40, 9], ctx + [1, 1, 40, 9])
    step([3, 1, 1, 1], [0, int(ctx[1]) + 1, int(ctx[2]) + 1, int(ctx[3]) + 1])  # the first ends
    step([0, 1, 1, 1], ctx + [0, 1, 1, 1])
    step([130, 1, 1, 20], ctx + [130, 1, 1, 20])  # and another begins in its place
    loop.ctx.copy_(dev(np.zeros(4, np.int32)))
    loop.new.zero_()
    loop.launch()
    assert int(loop.n_free.item()) == loop.pages and np.array_equal(loop.held.cpu().numpy(), [0] * 4)
    assert sorted(loop.free.cpu().numpy().tolist()) == list(range(loop.pages))


@pytest.mark.parametrize("bits", [8, 16])
def test_a_captured_step_replayed(qsa, bits):
    """The three calls and the lengths' growth as one graph, on a padded batch: the same bits as step by step."""
    results = []
    for captured in (False, True):
        rng = qi.rng_for(91, salt=bits)
        loop = Loop(qsa, rng, 5, 8, 2, 128, 16, 16, bits, pages=200, cols=30, max_rows=90)
        loop.new.copy_(dev(np.array([40, 3, 0, 17, 1], np.int32)))
        loop.x.copy_(dev(qi.normal_bf16(rng, (90, loop.width), 2.0)))
        loop.launch()
        loop.ctx.add_(loop.new)
        loop.new.copy_(dev(np.array([1, 1, 0, 1, 2], np.int32)))  # five rows of a batch of ninety
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                loop.launch()
                loop.ctx.add_(loop.new)
        got = []
        for _ in range(12):
            loop.x.copy_(dev(qi.normal_bf16(rng, (90, loop.width), 2.0)))
            if captured:
                graph.replay()
            else:
                loop.launch()
                loop.ctx.add_(loop.new)
            torch.cuda.synchronize()
            got += [loop.out.cpu().numpy().copy(), loop.lse.cpu().numpy().copy(), loop.table.cpu().numpy().copy()]
        assert qsa.qsa_read_status(loop.st) == (0, 0)
        results.append(got + [loop.k.cpu().numpy(), loop.v.cpu().numpy()])
    assert all(np.array_equal(a, b) for a, b in zip(*results))


def test_a_step_without_room_does_nothing(qsa):
    """Too few pages: the plan says so, and the calls behind it in the stream find no rows."""
    rng = qi.rng_for(92)
    loop = Loop(qsa, rng, 2, 8, 2, 128, 16, 16, 8, pages=6, cols=30, max_rows=90)
    loop.new.copy_(dev(np.array([60, 17], np.int32)))  # four pages and two
    loop.launch()
    loop.ctx.add_(loop.new)
    torch.cuda.synchronize()
    assert qsa.qsa_read_status(loop.st) == (0, 0) and int(loop.n_free.item()) == 0
    before = [t.clone() for t in (loop.k, loop.v, loop.ks, loop.vs, loop.table, loop.held, loop.out, loop.q)]
    loop.new.copy_(dev(np.array([1, 16], np.int32)))
    loop.launch()
    torch.cuda.synchronize()
    assert qsa.qsa_read_status(loop.st) == (qsa.QSA_ERR_NO_PAGES, 1)
    after = (loop.k, loop.v, loop.ks, loop.vs, loop.table, loop.held, loop.out, loop.q)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, after))
    assert int(loop.start.abs().max()) == 0
