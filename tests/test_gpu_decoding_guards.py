"""Out-of-bounds write checks of the drafted-tree and cache kernels, and calls
that overlap on the GPU.

Every buffer a call writes lies between two guard regions of a sentinel byte,
the workspace at exactly the size asked for.  The cases are ragged: empty
sequences, lengths around a tile, more sequences than threads of a CTA, head
counts of one and of many, windows, and a batch padded behind its last
sequence.  What a guarded call writes has to be the plain call's, bit by bit.
"""
import numpy as np
import pytest
import torch

import linear_attention_vlm_b200 as gdn

pytestmark = pytest.mark.gpu

GUARD, SENTINEL = 4096, 0xA5


class Guarded:
    def __init__(self, like=None, nbytes=0):
        dev = torch.device("cuda:0")
        n = like.numel() * like.element_size() if like is not None else nbytes
        self.raw = torch.full((GUARD + n + GUARD,), SENTINEL, dtype=torch.uint8, device=dev)
        self.t, self.n = self.raw[GUARD:GUARD + n], n
        if like is not None:
            self.t = self.t.view(like.dtype).view(like.shape)
            self.t.copy_(like)

    def check(self, want=None):
        torch.cuda.synchronize()
        assert bool((self.raw[:GUARD] == SENTINEL).all()) and bool((self.raw[GUARD + self.n:] == SENTINEL).all())
        if want is not None:
            assert torch.equal(self.t.view(torch.uint8), want.contiguous().view(torch.uint8))


def batch(ms, lens, cap, Hq, Hkv, pad, seed):
    gen = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    T, B = sum(ms) + pad, len(ms)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()      # noqa: E731
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()       # noqa: E731
    parents = [int(r.integers(-1, i)) if i else -1 for m in ms for i in range(m)] + [0] * pad
    pos = np.stack([[r.permutation(cap) for _ in range(Hkv)] for _ in range(B)])
    return dict(q=bf(T, Hq, 128), k=bf(T, Hkv, 128), v=bf(T, Hkv, 128), kc=bf(B, cap, Hkv, 128), vc=bf(B, cap, Hkv, 128),
                parents=ints(parents), cu=ints(np.cumsum([0] + list(ms))), lens=ints(lens), seen=ints([cap] * B), pos=ints(pos),
                w=torch.rand(B, Hkv, cap, generator=gen).cuda(), T=T, B=B, cap=cap, Hq=Hq, Hkv=Hkv, gen=gen)


CASES = [
    ([1], [1], 1, 1, 1, 0, 0),
    ([0, 1, 33, 64, 17], [0, 200, 129, 64, 1], 200, 16, 2, 5, 64),
    ([5, 0, 16], [77, 300, 300], 300, 24, 2, 0, 100),
    ([1] * 700, [i % 70 for i in range(700)], 69, 4, 2, 3, 0),
    ([3, 2], [5000, 4999], 5000, 40, 1, 1, 1000),
]


@pytest.mark.parametrize("ms,lens,cap,Hq,Hkv,pad,window", CASES, ids=range(len(CASES)))
def test_attention_and_weights_write_in_bounds(ms, lens, cap, Hq, Hkv, pad, window):
    c = batch(ms, lens, cap, Hq, Hkv, pad, cap)
    n = max(ms)
    ring = dict(cache_pos=c["pos"], seen=c["seen"], window=window) if window else {}
    o, lse = torch.full_like(c["q"], 3.0), torch.full((c["T"], Hq), 3.0, device="cuda")
    go, gl = Guarded(o), Guarded(lse)
    args = [c[x] for x in ("q", "k", "v", "parents", "kc", "vc", "lens", "cu")]
    gdn.gdn_tree_attention(*args, max_nodes=n, out=o, lse=lse, **ring)
    need = gdn.gdn_tree_attention_workspace_size(c["B"], c["T"], n, cap, Hq, Hkv)
    ws = Guarded(nbytes=need)
    gdn.gdn_tree_attention(*args, max_nodes=n, out=go.t, lse=gl.t, workspace=ws.t, **ring)
    go.check(o), gl.check(lse), ws.check()
    used = sum(ms)
    assert bool((o[used:] == 3.0).all()) and bool((lse[used:] == 3.0).all())
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())

    out, new = torch.full_like(c["w"], 7.0), torch.full((c["T"], Hkv), 7.0, device="cuda")
    gw, gn = Guarded(out), Guarded(new)
    ws = Guarded(nbytes=gdn.gdn_cache_weights_workspace_size(c["B"], c["T"], c["T"], cap, Hq, Hkv))
    args = [c["q"], lse, c["k"], c["kc"], c["w"], c["lens"], c["cu"], c["cu"]]
    gdn.gdn_cache_weights(*args, weights_out=out, new_weights=new, **ring)
    gdn.gdn_cache_weights(*args, weights_out=gw.t, new_weights=gn.t, workspace=ws.t, **ring)
    gw.check(out), gn.check(new), ws.check()
    empty = torch.arange(cap, device="cuda") >= c["lens"][:, None, None]
    assert bool((out == 7.0).logical_or(~empty).all()) and bool((new[used:] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ms,pad", [([1], 0), ([16, 0, 3], 2), ([32, 17], 1), ([64, 33, 0, 1], 5), ([2] * 300, 0)])
def test_step_writes_in_bounds(dtype, d, ms, pad):
    gen = torch.Generator().manual_seed(d)
    T, B, H = sum(ms) + pad, len(ms), 3
    mk = lambda *s: torch.randn(s, generator=gen)                                # noqa: E731
    q, k = (torch.nn.functional.normalize(mk(T, H, d), dim=-1).to(dtype).cuda() for _ in range(2))
    v, g, beta = mk(T, H, d).to(dtype).cuda(), -mk(T, H).abs().cuda(), torch.rand(T, H, generator=gen).cuda()
    cu = torch.tensor(np.cumsum([0] + ms), dtype=torch.int32).cuda()
    parents = torch.tensor([i // 2 - 1 for m in ms for i in range(m)] + [0] * pad, dtype=torch.int32).cuda()
    S = mk(B, H, d, d).cuda()
    out = torch.full_like(v, 3.0)
    go, gs = Guarded(out), Guarded(S)
    gdn.gdn_tree_step(q, k, v, g, beta, parents, S, cu, out=out)
    gdn.gdn_tree_step(q, k, v, g, beta, parents, gs.t, cu, out=go.t)
    go.check(out), gs.check(S)
    assert bool(torch.isfinite(out.float()).all()) and bool((out[sum(ms):] == 3.0).all())


@pytest.mark.parametrize("ms,lens,cap,Hkv,recent,pad", [
    ([1], [1], 1, 1, 0, 0),
    ([4, 0, 9], [50, 50, 13], 50, 2, 10, 3),
    ([500, 3], [40, 40], 40, 9, 40, 0),
    ([2] * 90, [33] * 90, 33, 4, 5, 1),
    ([30000], [0], 700, 2, 100, 0),
    ([20000, 1], [11000, 11000], 11000, 2, 64, 7),
])
def test_insert_writes_in_bounds(ms, lens, cap, Hkv, recent, pad):
    c = batch(ms, lens, cap, Hkv, Hkv, pad, cap + Hkv)
    nw = torch.rand(c["T"], Hkv, generator=c["gen"]).cuda()
    slots = torch.full((c["T"], Hkv), -7, dtype=torch.int32, device="cuda")
    plain = [c["kc"].clone(), c["vc"].clone(), c["w"].clone(), c["pos"].clone(), c["lens"].clone(), c["seen"].clone(), slots]
    guarded = [Guarded(x) for x in plain]
    need = gdn.gdn_cache_insert_workspace_size(c["B"], c["T"], cap, Hkv, 128)
    ws = Guarded(nbytes=need)
    for k_c, v_c, w, pos, ln, sn, sl, scratch in (plain + [None], [x.t for x in guarded] + [ws.t]):
        gdn.gdn_cache_insert(c["k"], c["v"], k_c, v_c, w, pos, ln, sn, c["cu"], recent=recent, new_weights=nw, slots=sl,
                             workspace=scratch)
    for x, y in zip(guarded, plain):
        x.check(y)
    ws.check()
    assert bool((slots[sum(ms):] == -7).all())
    assert plain[4].tolist() == [min(cap, n + m) for n, m in zip(lens, ms)]


def test_overlapping_calls_with_a_workspace_each():
    """Four streams at once, a dozen calls each: every result is the one of a
    call on its own."""
    sets = [batch([3, 1, 20], [900, 1000, 0], 1000, 16, 2, 0, s) for s in range(4)]
    def turn(c, o, l):
        gdn.gdn_tree_attention(c["q"], c["k"], c["v"], c["parents"], c["kc"], c["vc"], c["lens"], c["cu"], max_nodes=20, out=o, lse=l)
        w, new = gdn.gdn_cache_weights(c["q"], l, c["k"], c["kc"], c["w"], c["lens"], c["cu"], c["cu"],
                                       weights_out=torch.zeros_like(c["w"]))
        got = gdn.gdn_cache_insert(c["k"], c["v"], c["kc"].clone(), c["vc"].clone(), w, c["pos"], c["lens"], c["seen"], c["cu"],
                                   recent=50, new_weights=new, weights_out=torch.zeros_like(w), pos_out=torch.zeros_like(c["pos"]),
                                   lens_out=torch.zeros_like(c["lens"]), seen_out=torch.zeros_like(c["seen"]))
        return [o, l, w, new] + list(got)
    fresh = lambda c: (torch.empty_like(c["q"]), torch.empty(c["T"], 16, device="cuda"))  # noqa: E731
    alone = []
    for c in sets:
        alone.append([x.clone() for x in turn(c, *fresh(c))])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[] for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(12):
        for s, c, o in zip(streams, sets, outs):
            with torch.cuda.stream(s):
                o.append(turn(c, *fresh(c)))
    torch.cuda.synchronize()
    for want, o in zip(alone, outs):
        for got in o:
            assert all(torch.equal(a, b) for a, b in zip(want, got))
