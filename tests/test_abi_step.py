"""Host-only refusals of the step operators: no GPU, no launch (the dangling pointers are
never read).  Each group first makes the same call with an empty extent, which must be
QSA_OK."""
import ctypes

import pytest

A, B, U = 0x10000, 0x20000, 0x10002   # aligned, aligned, misaligned


@pytest.fixture(scope="module")
def qsa():
    import __graft_entry__

    __graft_entry__.build()
    import sparse_attention_token_qsa_gb300 as m

    return m


@pytest.fixture(scope="module")
def lib(qsa):
    return qsa.library()


def P(x):
    return ctypes.c_void_p(x or 0)


def plan(lib, **kw):
    a = dict(ctx=B, new=B, n=3, page=16, pages=100, table=B, tl=40, tc=40, held=B, ho=B, free=B, nf=B, nfo=B, rows=9, start=B, slot=B,
             pos=B, seq=B, st=B)
    a.update(kw)
    return lib.qsa_page_plan(P(a["ctx"]), P(a["new"]), a["n"], a["page"], a["pages"], P(a["table"]), a["tl"], a["tc"], P(a["held"]),
                             P(a["ho"]), P(a["free"]), P(a["nf"]), P(a["nfo"]), a["rows"], P(a["start"]), P(a["slot"]),
                             P(a["pos"]), P(a["seq"]), P(a["st"]), None)


def test_plan_refusals(lib):
    assert plan(lib, n=0) == 0 and plan(lib, n=0, ctx=0, table=0, st=0, page=0) == 0
    for kw in (dict(ctx=0), dict(new=0), dict(table=0), dict(held=0), dict(ho=0), dict(free=0), dict(nf=0), dict(nfo=0),
               dict(start=0), dict(slot=0), dict(st=0), dict(n=-1), dict(page=0), dict(page=-1), dict(pages=0), dict(pages=-1),
               dict(tl=0), dict(tl=-1), dict(tc=39), dict(tc=0), dict(tc=-1), dict(rows=-1), dict(n=65536), dict(pages=1 << 27),
               dict(tl=1 << 27, tc=1 << 27)):
        assert plan(lib, **kw) == 1, kw
    assert plan(lib, n=0, rows=-1) == 1


def write(lib, **kw):
    a = dict(q=A, qs=5120, nq=16, k=A, ks=5120, v=A, vs=5120, nkv=2, hd=256, qw=A, kw=A, eps=1e-6, cos=A, sin=A, tr=100, pos=B, ctx=B,
             start=B, n=2, rows=9, kp=A, vp=A, ksc=B, vsc=B, unit=16, pages=100, page=16, table=B, tl=40, tc=40, out=A, os=4096, st=B)
    a.update(kw)
    return lib.qsa_qkv_write(P(a["q"]), a["qs"], a["nq"], P(a["k"]), a["ks"], P(a["v"]), a["vs"], a["nkv"], a["hd"], P(a["qw"]),
                             P(a["kw"]), a["eps"], P(a["cos"]), P(a["sin"]), a["tr"], P(a["pos"]), P(a["ctx"]), P(a["start"]),
                             a["n"], a["rows"], P(a["kp"]), P(a["vp"]), P(a["ksc"]), P(a["vsc"]), a["unit"], a["pages"],
                             a["page"], P(a["table"]), a["tl"], a["tc"], P(a["out"]), a["os"], P(a["st"]), None)


SHARED = [dict(q=0), dict(q=U), dict(table=0), dict(ctx=0), dict(start=0), dict(st=0), dict(qs=4088), dict(qs=5124), dict(qs=-8),
          dict(nq=0), dict(nkv=0), dict(nkv=-2), dict(nq=15), dict(hd=64), dict(hd=192), dict(pages=0), dict(pages=-1),
          dict(page=0), dict(page=-16), dict(tl=0), dict(tl=-1), dict(tc=39), dict(tc=-1), dict(pages=1 << 27),
          dict(tl=1 << 27, tc=1 << 27), dict(n=65536), dict(rows=1 << 28), dict(n=-1), dict(rows=-1), dict(unit=0), dict(unit=8),
          dict(unit=24), dict(unit=256, page=256), dict(unit=32), dict(unit=16, page=40), dict(os=4088), dict(os=4100),
          dict(os=-8), dict(out=0), dict(out=U)]


def test_write_refusals(lib):
    assert write(lib, n=0) == 0 and write(lib, rows=0) == 0 and write(lib, n=0, q=0, kp=0, table=0) == 0
    for kw in SHARED:
        assert write(lib, **kw) == 1, kw
    for kw in (dict(k=0), dict(k=U), dict(v=0), dict(v=U), dict(kp=0), dict(kp=U), dict(vp=0), dict(vp=U), dict(ks=504), dict(ks=516),
               dict(vs=504), dict(vs=-8), dict(qw=U), dict(kw=U), dict(cos=0), dict(sin=0), dict(cos=U), dict(sin=U), dict(tr=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(ksc=0), dict(vsc=0), dict(tc=0)):
        assert write(lib, **kw) == 1, kw
    assert write(lib, n=0, eps=-1.0) == 1


def attend(lib, **kw):
    a = dict(q=A, qs=4096, nq=16, nkv=2, hd=256, k=A, v=A, ks=B, vs=B, unit=16, pages=100, page=16, table=B, tl=40, tc=40, ctx=B,
             start=B, n=2, rows=9, mask=B, words=1, first=4, window=64, scale=0.0625, out=A, os=4096, lse=B, st=B, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.qsa_cache8_attn(P(a["q"]), a["qs"], a["nq"], a["nkv"], a["hd"], P(a["k"]), P(a["v"]), P(a["ks"]), P(a["vs"]), a["unit"],
                               a["pages"], a["page"], P(a["table"]), a["tl"], a["tc"], P(a["ctx"]), P(a["start"]), a["n"],
                               a["rows"], P(a["mask"]), a["words"], a["first"], a["window"], a["scale"], P(a["out"]), a["os"],
                               P(a["lse"]), P(a["st"]), P(a["ws"]), a["wsb"], None)


def test_attend_refusals(lib):
    assert attend(lib, n=0) == 0 and attend(lib, rows=0) == 0 and attend(lib, n=0, q=0, k=0, table=0, ws=0) == 0
    for kw in SHARED:
        assert attend(lib, **{k: (v - 1024 if k == "qs" and v == 5124 else v) for k, v in kw.items()}) == 1, kw
    for kw in (dict(k=0), dict(k=U), dict(v=0), dict(v=U), dict(ks=0), dict(vs=0), dict(words=0), dict(words=-1), dict(first=-1),
               dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=0), dict(ws=U), dict(wsb=-1),
               dict(wsb=lib.qsa_cache8_workspace_bytes(2, 9, 16, 2, 256) - 1)):
        assert attend(lib, **kw) == 1, kw
    assert attend(lib, n=0, window=-1) == 1


def test_attend_workspace_bytes(lib, qsa):
    f = lib.qsa_cache8_workspace_bytes
    for bad in ((-1, 1, 16, 2, 256), (1, -1, 16, 2, 256), (1, 1, 0, 2, 256), (1, 1, 16, 0, 256), (1, 1, 15, 2, 256), (1, 1, 16, 2, 64)):
        assert f(*bad) == -1
        with pytest.raises(ValueError):
            qsa.new_cache8_workspace(*bad, device="cpu")
    for n in (1, 31, 33, 600):
        for rows in (1, 4, 40, 1000):
            for group in (1, 4, 8, 130):
                for hd in (128, 256):
                    here = f(n, rows, group, 1, hd)
                    assert here > 0 and here == f(n, rows, 8 * group, 8, hd)
                    assert here <= min(f(n + 1, rows, group, 1, hd), f(n, rows + 1, group, 1, hd), f(n, rows, group + 1, 1, hd),
                                       f(n, rows, group, 1, 256))
    assert qsa.new_cache8_workspace(3, 9, 16, 2, 256, device="cpu").numel() == f(3, 9, 16, 2, 256)


def test_status_of_too_few_pages(qsa):
    assert "pages" in qsa.status_string(qsa.QSA_ERR_NO_PAGES)


def test_binding_refuses_host_tensors(qsa):
    import torch

    x = torch.zeros(8)
    with pytest.raises(ValueError):
        qsa.qsa_page_plan(x, x, 1, 16, 1, x, 1, 1, x, x, x, x, x, 1, x, x, x, x, x)
    with pytest.raises(ValueError):
        qsa.qsa_cache8_attn(x, 128, 1, 1, 128, x, x, x, x, 16, 1, 16, x, 1, 1, x, x, 1, 1, None, 0, 0, 0, 1.0, x, 128, x, x, x)
    with pytest.raises(TypeError):
        qsa.qsa_qkv_write([1], 128, 1, x, 128, x, 128, 1, 128, x, x, 0.0, x, x, 1, x, x, x, 1, 1, x, x, x, x, 16, 1, 16, x, 1, 1, x, 128, x)
