"""Calls over drafted trees and a bounded cache that the header allows and the
parity tests do not make: optional pointers left out, a cache of no slots,
insertions and steps captured into a graph and replayed."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_vlm_b200 as gdn
from oracle import decoding as D

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def np64(x):
    return x.detach().to("cpu", torch.float64).numpy()


def mk(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen).to(dtype).cuda()


@pytest.mark.parametrize("n", [3, 40])
def test_no_log_sum_exp_wanted(n):
    gen = torch.Generator().manual_seed(n)
    q, k, v, kc, vc = mk(gen, n, 16, 128), mk(gen, n, 2, 128), mk(gen, n, 2, 128), mk(gen, 1, 900, 2, 128), mk(gen, 1, 900, 2, 128)
    lens = ints([877])
    o, _ = gdn.gdn_tree_attention(q, k, v, None, kc, vc, lens, max_nodes=n)
    ws = torch.empty(gdn.gdn_tree_attention_workspace_size(1, n, n, 900, 16, 2), dtype=torch.uint8, device="cuda")
    got = torch.empty_like(o)
    st = gdn.library().gdn_tree_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, kc.data_ptr(), vc.data_ptr(),
                                          lens.data_ptr(), None, None, got.data_ptr(), None, 1, n, n, 900, 16, 2, 128, 0,
                                          ctypes.c_float(0.0), 1, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(got, o)


@pytest.mark.parametrize("dtype,code", [(torch.float32, 0), (torch.bfloat16, 1)])
def test_no_state_is_a_state_of_zeros(dtype, code):
    gen = torch.Generator().manual_seed(0)
    q, k, v = (mk(gen, 10, 3, 64, dtype=dtype) * 0.2 for _ in range(3))
    g, beta = -torch.rand(10, 3, generator=gen).cuda(), torch.rand(10, 3, generator=gen).cuda()
    want = gdn.gdn_tree_step(q, k, v, g, beta, None, torch.zeros(2, 3, 64, 64).cuda())
    got = torch.empty_like(want)
    st = gdn.library().gdn_tree_step(*[ctypes.c_void_p(x.data_ptr()) if x.dtype != torch.float32 or i < 3 else
                                       ctypes.cast(x.data_ptr(), ctypes.POINTER(ctypes.c_float)) for i, x in enumerate((q, k, v, g, beta))],
                                     None, None, got.data_ptr(), None, 2, 10, 5, 3, 64, 64, code, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(got, want)


def test_a_cache_of_no_slots():
    # 1e-3 bounds the error of the scores, 2^-23 128 |q| |k| / sqrt(128) for rows of norm up to 16
    gen = torch.Generator().manual_seed(1)
    q, k, v = mk(gen, 7, 4, 128), mk(gen, 7, 2, 128), mk(gen, 7, 2, 128)
    none, lens, cu, parents = torch.empty(2, 0, 2, 128, dtype=torch.bfloat16, device="cuda"), ints([0, 0]), [0, 5, 7], [-1, 0, 0, 2, -1, -1, 0]
    o, lse = gdn.gdn_tree_attention(q, k, v, ints(parents), none, none, lens, ints(cu), window=3)
    ref, ref_lse = D.tree_attention(np64(q), np64(k), np64(v), parents, np64(none), np64(none), [0, 0], cu, window=3)
    assert np.all(np.abs(np64(o) - ref) <= 2.0 ** -8 * (np.abs(ref) + np.abs(np64(v)).max()) + 1e-3)
    assert np.abs(np64(lse) - ref_lse).max() <= 1e-3
    w = torch.empty(2, 2, 0, device="cuda")
    _, new = gdn.gdn_cache_weights(q, lse, k, none, w, lens, ints(cu), ints(cu), window=3)
    _, ref_new = D.cache_weights(np64(q), np64(lse), np64(k), np64(none), np64(w), [0, 0], cu, cu, window=3)
    assert np.allclose(np64(new), ref_new, rtol=1e-3, atol=1e-6)


@pytest.mark.parametrize("B,Hkv,m,cap", [(3, 2, 4, 300), (1, 9, 30, 300), (2, 1, 900, 11000), (90, 2, 40, 64)])
def test_insertions_and_steps_in_a_graph(B, Hkv, m, cap):
    """In place, over and over: replays are what as many calls are, also after
    the lists' lengths have changed on the device."""
    gen = torch.Generator().manual_seed(B + m)
    T = B * m
    k, v = mk(gen, T, Hkv, 64), mk(gen, T, Hkv, 64)
    kc, vc = mk(gen, B, cap, Hkv, 64), mk(gen, B, cap, Hkv, 64)
    w, nw = torch.rand(B, Hkv, cap, generator=gen).cuda(), torch.rand(T, Hkv, generator=gen).cuda()
    pos = torch.arange(cap, dtype=torch.int32).expand(B, Hkv, cap).contiguous().cuda()
    cu = ints(np.arange(B + 1) * m)
    n = min(m, 20)
    q, kk, vv = (mk(gen, B * n, 2, 64) * 0.1 for _ in range(3))
    g, beta, S = -torch.rand(B * n, 2, generator=gen).cuda(), torch.rand(B * n, 2, generator=gen).cuda(), torch.randn(B, 2, 64, 64, generator=gen).cuda()

    def state():
        return [kc.clone(), vc.clone(), w.clone(), pos.clone(), ints([max(0, cap - 7 * b) for b in range(B)]), ints([cap + b for b in range(B)])]

    def call(s, slots, out):
        gdn.gdn_cache_insert(k, v, s[0], s[1], s[2], s[3], s[4], s[5], cu, recent=cap // 10, new_weights=nw, slots=slots)
        gdn.gdn_tree_step(q, kk, vv, g, beta, None, S, out=out)

    def outputs():
        return torch.zeros(T, Hkv, dtype=torch.int32, device="cuda"), torch.zeros_like(vv)

    warm = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(warm, *outputs())
    torch.cuda.current_stream().wait_stream(side)
    a, b, oa, ob = state(), state(), outputs(), outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, *oa)
    for turn in range(4):
        if turn == 2:
            lens = [(3 * b_) % (m + 1) for b_ in range(B)]
            cu.copy_(ints(np.concatenate([[0], np.cumsum(lens)])))
        graph.replay()
        call(b, *ob)
        torch.cuda.synchronize()
        for x, y in zip(a + list(oa), b + list(ob)):
            assert torch.equal(x, y)
