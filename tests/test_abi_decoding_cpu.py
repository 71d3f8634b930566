"""Refusals of the entry points over drafted trees and a bounded cache: wrong
arguments are turned away on the host, before anything is enqueued."""
import ctypes

import pytest
import torch

import linear_attention_vlm_b200 as gdn
from linear_attention_vlm_b200 import gdn as binding

INV, UNS, WS, OK = (binding.GDN_ERR_INVALID_ARG, binding.GDN_ERR_UNSUPPORTED, binding.GDN_ERR_WORKSPACE, binding.GDN_OK)
M = 1 << 24     # spacing of the made-up addresses


@pytest.fixture(scope="module")
def lib():
    return gdn.library()


def attention(lib, **kw):
    a = dict(q=1 * M, k=2 * M, v=3 * M, parents=4 * M, cu=5 * M, kc=6 * M, vc=7 * M, lens=8 * M, pos=None, seen=None,
             o=9 * M, lse=10 * M, B=2, T=8, n=8, cap=64, Hq=4, Hkv=2, d=128, window=0, scale=0.0, dtype=1, ws=11 * M,
             wsb=1 << 40)
    a.update(kw)
    return lib.gdn_tree_attention(a["q"], a["k"], a["v"], a["parents"], a["cu"], a["kc"], a["vc"], a["lens"], a["pos"],
                                  a["seen"], a["o"], a["lse"], a["B"], a["T"], a["n"], a["cap"], a["Hq"], a["Hkv"],
                                  a["d"], a["window"], ctypes.c_float(a["scale"]), a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(o=None), INV), (dict(lens=None), INV),
    (dict(kc=None), INV), (dict(vc=None), INV), (dict(q=M + 8), INV), (dict(parents=4 * M + 4), INV),
    (dict(lse=10 * M + 4), INV), (dict(B=0), INV), (dict(T=-1), INV), (dict(cap=-1), INV), (dict(n=0), INV),
    (dict(n=65), INV), (dict(Hq=5), INV), (dict(Hkv=0), INV), (dict(window=-1), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(dtype=7), INV), (dict(pos=12 * M), INV),
    (dict(cu=None, T=9), INV), (dict(cu=None, T=40, n=8), INV), (dict(cap=1 << 31), INV), (dict(B=4, cap=1 << 30), INV),
    (dict(T=1 << 31), INV), (dict(B=70000), INV),
    (dict(d=64), UNS), (dict(dtype=0), UNS), (dict(Hq=258, Hkv=2), UNS), (dict(ws=None), WS), (dict(wsb=8), WS),
    (dict(o=1 * M), INV), (dict(o=2 * M + 1024), INV), (dict(lse=9 * M + 16), INV), (dict(ws=6 * M), INV),
    (dict(lse=8 * M), INV), (dict(T=0), OK),
])
def test_tree_attention_refuses(lib, kw, status):
    assert attention(lib, **kw) == status


def test_workspace_sizes_are_host_arithmetic():
    assert gdn.gdn_tree_attention_workspace_size(1, 1, 1, 8192, 16, 2) > 0
    assert gdn.gdn_tree_attention_workspace_size(1, 1, 65, 8192, 16, 2) == 0
    assert gdn.gdn_tree_attention_workspace_size(1, 1, 1, 8192, 16, 3) == 0
    assert gdn.gdn_tree_attention_workspace_size(1, 1, 1, 8192, 16, 2, d=64) == 0
    assert gdn.gdn_cache_weights_workspace_size(1, 1, 1, 8192, 16, 2) > 0
    assert gdn.gdn_cache_weights_workspace_size(1, -1, 1, 8192, 16, 2) == 0
    assert gdn.library().gdn_cache_insert_workspace_size(1, 8, 0, 2, 128, 1) == 0
    assert gdn.library().gdn_cache_insert_workspace_size(1, 8, 16, 2, 128, 1) > 0


def step(lib, **kw):
    a = dict(q=1 * M, k=2 * M, v=3 * M, g=4 * M, beta=5 * M, parents=6 * M, state=7 * M, out=8 * M, cu=9 * M, B=2, T=8,
             n=8, H=2, dk=64, dv=64, dtype=1)
    a.update(kw)
    return lib.gdn_tree_step(a["q"], a["k"], a["v"], a["g"], a["beta"], a["parents"], a["state"], a["out"], a["cu"],
                             a["B"], a["T"], a["n"], a["H"], a["dk"], a["dv"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(out=None), INV), (dict(g=None), INV), (dict(k=2 * M + 4), INV), (dict(B=0), INV),
    (dict(T=-1), INV), (dict(H=0), INV), (dict(n=0), INV), (dict(n=65), INV), (dict(dtype=5), INV),
    (dict(cu=None, T=9), INV), (dict(cu=None, T=40, n=8), INV), (dict(out=3 * M), INV), (dict(out=7 * M + 64), INV),
    (dict(dk=96, dv=96), UNS), (dict(dk=128, dv=64), UNS), (dict(T=0), OK),
])
def test_tree_step_refuses(lib, kw, status):
    assert step(lib, **kw) == status


def weights(lib, **kw):
    a = dict(q=1 * M, lse=2 * M, k=3 * M, kc=4 * M, wi=5 * M, wo=5 * M, wn=6 * M, cuq=7 * M, cut=8 * M, lens=9 * M,
             pos=None, seen=None, B=2, Tq=4, T=8, cap=64, Hq=4, Hkv=2, d=128, window=0, scale=0.0, dtype=1, ws=10 * M,
             wsb=1 << 40)
    a.update(kw)
    return lib.gdn_cache_weights(a["q"], a["lse"], a["k"], a["kc"], a["wi"], a["wo"], a["wn"], a["cuq"], a["cut"],
                                 a["lens"], a["pos"], a["seen"], a["B"], a["Tq"], a["T"], a["cap"], a["Hq"], a["Hkv"],
                                 a["d"], a["window"], ctypes.c_float(a["scale"]), a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(lse=None), INV), (dict(k=None), INV), (dict(kc=None), INV), (dict(wi=None), INV),
    (dict(wo=None), INV), (dict(wn=None), INV), (dict(lens=None), INV), (dict(q=M + 8), INV), (dict(cuq=None), INV),
    (dict(cut=None), INV), (dict(cuq=None, cut=None, Tq=3), INV), (dict(pos=11 * M), INV), (dict(B=0), INV),
    (dict(window=-2), INV), (dict(wo=5 * M + 64), INV), (dict(wn=5 * M), INV), (dict(wo=4 * M), INV),
    (dict(d=64), UNS), (dict(dtype=0), UNS), (dict(wsb=0), WS), (dict(T=0, Tq=0, cap=0), OK),
])
def test_cache_weights_refuses(lib, kw, status):
    assert weights(lib, **kw) == status


def insert(lib, **kw):
    a = dict(k=1 * M, v=2 * M, kc=3 * M, vc=4 * M, wi=5 * M, wo=5 * M, pi=6 * M, po=6 * M, li=7 * M, lo=7 * M, si=8 * M,
             so=8 * M, wn=9 * M, slots=10 * M, cu=11 * M, B=2, T=8, cap=64, Hkv=2, d=128, recent=0, dtype=1, ws=12 * M,
             wsb=1 << 40)
    a.update(kw)
    return lib.gdn_cache_insert(a["k"], a["v"], a["kc"], a["vc"], a["wi"], a["wo"], a["pi"], a["po"], a["li"], a["lo"],
                                a["si"], a["so"], a["wn"], a["slots"], a["cu"], a["B"], a["T"], a["cap"], a["Hkv"],
                                a["d"], a["recent"], a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(kc=None), INV), (dict(vc=None), INV), (dict(wi=None), INV),
    (dict(po=None), INV), (dict(lo=None), INV), (dict(si=None), INV), (dict(slots=None), INV), (dict(kc=3 * M + 8), INV),
    (dict(B=0), INV), (dict(T=-1), INV), (dict(cap=0), INV), (dict(recent=-1), INV), (dict(recent=65), INV),
    (dict(dtype=4), INV), (dict(cu=None, T=9), INV), (dict(B=40000), INV), (dict(cap=1 << 30), INV),
    (dict(d=4), UNS), (dict(ws=None), WS), (dict(wsb=16), WS), (dict(vc=3 * M + 64), INV), (dict(kc=1 * M), INV),
    (dict(wo=5 * M + 16), INV), (dict(po=5 * M), INV), (dict(lo=8 * M), INV), (dict(slots=9 * M), INV),
])
def test_cache_insert_refuses(lib, kw, status):
    assert insert(lib, **kw) == status


def test_binding_refuses_cpu_tensors():
    x, s = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, 2)
    c = torch.zeros(1, 8, 2, 128, dtype=torch.bfloat16)
    one, w = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 8)
    with pytest.raises(ValueError):
        gdn.gdn_tree_attention(x, x, x, None, c, c, one)
    with pytest.raises(ValueError):
        gdn.gdn_tree_step(x, x, x, s, s, None, torch.zeros(1, 2, 128, 128))
    with pytest.raises(ValueError):
        gdn.gdn_cache_weights(x, s, x, c, w, one)
    with pytest.raises(ValueError):
        gdn.gdn_cache_insert(x, x, c, c, w, w.int(), one, one)
