"""Host-only refusals of the cache operators: no GPU, no launch (the dangling
pointers are never read).  Each group first makes the same call with an empty
extent, which must be QSA_OK."""
import ctypes

import pytest

A, B, U = 0x10000, 0x20000, 0x10002   # aligned, aligned, misaligned


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    import sparse_attention_token_qsa_gb300 as qsa

    return qsa.library()


def P(x):
    return ctypes.c_void_p(x or 0)


def tree(lib, **kw):
    a = dict(q=A, qs=4096, nq=16, nkv=2, hd=256, k=A, v=A, pages=100, page=16, table=B, tl=40, tc=40, ctx=B, start=B, n=2,
             rows=9, mask=B, words=1, scale=0.0625, out=A, os=4096, lse=B, st=B, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.qsa_tree_attn(P(a["q"]), a["qs"], a["nq"], a["nkv"], a["hd"], P(a["k"]), P(a["v"]), a["pages"], a["page"],
                             P(a["table"]), a["tl"], a["tc"], P(a["ctx"]), P(a["start"]), a["n"], a["rows"], P(a["mask"]),
                             a["words"], a["scale"], P(a["out"]), a["os"], P(a["lse"]), P(a["st"]), P(a["ws"]), a["wsb"], None)


def mass(lib, **kw):
    a = dict(q=A, qs=4096, nq=16, nkv=2, hd=256, k=A, pages=100, page=16, table=B, tl=40, tc=40, ctx=B, start=B, n=2,
             rows=9, mask=B, words=1, scale=0.0625, lse=B, w=0, carry=1.0, mass=A, cols=640, st=B)
    a.update(kw)
    return lib.qsa_attn_mass(P(a["q"]), a["qs"], a["nq"], a["nkv"], a["hd"], P(a["k"]), a["pages"], a["page"], P(a["table"]),
                             a["tl"], a["tc"], P(a["ctx"]), P(a["start"]), a["n"], a["rows"], P(a["mask"]), a["words"],
                             a["scale"], P(a["lse"]), P(a["w"]), a["carry"], P(a["mass"]), a["cols"], P(a["st"]), None)


SHARED = [dict(q=0), dict(q=U), dict(k=0), dict(k=U), dict(table=0), dict(ctx=0), dict(start=0), dict(st=0), dict(qs=4088),
          dict(qs=4100), dict(qs=-8), dict(nq=0), dict(nkv=0), dict(nkv=-2), dict(nq=15), dict(hd=64), dict(hd=192),
          dict(pages=0), dict(pages=-1), dict(page=0), dict(page=-16), dict(tl=0), dict(tl=-1), dict(tc=39), dict(tc=-1),
          dict(words=0), dict(words=-1), dict(scale=float("nan")), dict(scale=float("inf")),
          dict(pages=1 << 27), dict(tl=1 << 27, tc=1 << 27), dict(n=65536), dict(rows=1 << 28), dict(n=-1), dict(rows=-1)]


@pytest.mark.parametrize("fn", [tree, mass])
def test_attention_refusals(lib, fn):
    assert fn(lib, n=0) == 0 and fn(lib, rows=0) == 0
    assert fn(lib, n=0, q=0, k=0, table=0) == 0
    for kw in SHARED:
        assert fn(lib, **kw) == 1, kw
    assert fn(lib, n=0, words=-1) == 1 and fn(lib, rows=0, tl=-1) == 1


def test_tree_refusals(lib):
    for kw in (dict(v=0), dict(v=U), dict(out=0), dict(out=U), dict(os=4088), dict(os=4100), dict(os=-8), dict(ws=0), dict(ws=U),
               dict(wsb=-1), dict(wsb=lib.qsa_tree_workspace_bytes(2, 9, 16, 2, 256) - 1)):
        assert tree(lib, **kw) == 1, kw


def test_tree_workspace_bytes(lib):
    f = lib.qsa_tree_workspace_bytes
    for bad in ((-1, 1, 16, 2, 256), (1, -1, 16, 2, 256), (1, 1, 0, 2, 256), (1, 1, 16, 0, 256), (1, 1, 15, 2, 256),
                (1, 1, 16, 2, 64)):
        assert f(*bad) == -1
    assert f(1, 1, 16, 2, 256) > 0 and f(0, 0, 16, 2, 256) >= 0
    # grows with each extent: a workspace for the largest call serves every smaller one
    assert f(2, 9, 16, 2, 256) <= f(3, 9, 16, 2, 256) <= f(3, 64, 16, 2, 256)


def test_mass_refusals(lib):
    for kw in (dict(lse=0), dict(mass=0), dict(mass=U), dict(cols=642), dict(cols=-4), dict(carry=-0.5),
               dict(carry=float("nan")), dict(carry=float("inf"))):
        assert mass(lib, **kw) == 1, kw
    assert mass(lib, n=0, carry=-1.0) == 1


def evict(lib, **kw):
    a = dict(m=A, cols=1024, nkv=2, ln=B, n=3, tokens=1000, keep=256, first=4, last=64, unit=4, sel=B, sc=259, ns=B, st=B)
    a.update(kw)
    return lib.qsa_evict_select(P(a["m"]), a["cols"], a["nkv"], P(a["ln"]), a["n"], a["tokens"], a["keep"], a["first"],
                                a["last"], a["unit"], P(a["sel"]), a["sc"], P(a["ns"]), P(a["st"]), None)


def test_evict_refusals(lib):
    assert evict(lib, n=0) == 0 and evict(lib, n=0, m=0, ln=0, sel=0) == 0
    for kw in (dict(m=0), dict(m=U), dict(cols=996), dict(cols=1022), dict(nkv=0), dict(ln=0), dict(sel=0), dict(ns=0),
               dict(st=0), dict(sc=258), dict(keep=0), dict(keep=-4), dict(keep=255), dict(unit=2), dict(unit=0), dict(unit=-1),
               dict(first=3), dict(last=2), dict(first=-4), dict(last=-4), dict(first=200, last=60), dict(n=-1),
               dict(tokens=-1), dict(n=(1 << 20) + 1), dict(tokens=2 ** 31 - 1, cols=1 << 31)):
        assert evict(lib, **kw) == 1, kw
    assert evict(lib, n=0, unit=3) == 1


def compact(lib, **kw):
    a = dict(k=A, v=A, width=512, pages=100, table=B, tl=40, tc=40, page=16, keep=B, kc=300, nk=B, n=3, most=259, first=0, m=B,
             cols=640, nkv=2, bk=A, kb=B, st=B)
    a.update(kw)
    return lib.qsa_cache_compact(P(a["k"]), P(a["v"]), a["width"], a["pages"], P(a["table"]), a["tl"], a["tc"], a["page"],
                                 P(a["keep"]), a["kc"], P(a["nk"]), a["n"], a["most"], P(a["first"]), P(a["m"]), a["cols"],
                                 a["nkv"], P(a["bk"]), P(a["kb"]), P(a["st"]), None)


def test_compact_refusals(lib):
    assert compact(lib, n=0) == 0 and compact(lib, most=0) == 0 and compact(lib, n=0, k=0, keep=0) == 0
    for kw in (dict(k=0), dict(k=U), dict(v=0), dict(v=U), dict(width=0), dict(width=516), dict(width=-8), dict(pages=-1),
               dict(table=0), dict(tl=-1), dict(tc=39), dict(tc=0), dict(page=0), dict(keep=0), dict(kc=258), dict(nk=0),
               dict(n=-1), dict(most=-1), dict(cols=-1), dict(nkv=0), dict(nkv=-1), dict(bk=U), dict(kb=0), dict(st=0),
               dict(n=65536), dict(width=(1 << 24) + 8), dict(tl=1 << 28, tc=1 << 28), dict(pages=1 << 27)):
        assert compact(lib, **kw) == 1, kw


def test_binding_refuses_host_tensors():
    import torch

    import sparse_attention_token_qsa_gb300 as qsa

    x = torch.zeros(8)
    with pytest.raises(ValueError):
        qsa.qsa_evict_select(x, 8, 1, x, 1, 8, 4, 0, 0, 4, x, 8, x, x)
    with pytest.raises(TypeError):
        qsa.qsa_attn_mass([1], 128, 1, 1, 128, x, 1, 1, x, 1, 1, x, x, 1, 1, None, 0, 1.0, x, None, 1.0, x, 8, x)
