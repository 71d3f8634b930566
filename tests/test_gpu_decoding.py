"""Parity of the operators over drafted trees and a bounded cache with the
fp64 oracle, through the C ABI.

Bars.  bf16 rounding is off by at most 2^-8 relative.
Attention output: |o - ref| <= 2^-8 |ref| + 2^-8 max|v| (the rounding of o, and
of the probabilities in a weighted mean of values up to max|v|), the bar of
gdn_swa_attention; plus, for both, what an error E of the scores makes of
them (a relative error of exp).
E: a score is a sum of d products added in fp32, each addition off by at most
2^-23 of the sum of magnitudes (the tensor core may cut instead of rounding), so
E = 2^-23 d scale max sum|q k|; lse adds the error of its sum of L positive
terms, <= (L/64 + 64) 2^-23 relative for sums of 64 at a time, and 8 steps
2^-23 of its own size and of the exponential.
Weights: every term is off by E and by the fp32 difference score - lse, so
|w - ref| <= ref (E + 2^-22 (8 + max(|score|, |lse|)) + rows 2^-23) + 2^-23 |ref + w_in|.
Tree step: fp32 within 1e-4 of the largest value, the bar of gdn_prefill; bf16
2^-8 |ref| for the rounding of the output plus 7e-4 of the largest |S row| or |v|
(64 nodes deep, each a sum of up to 192 fp32 products of at most that size:
64 * 192 * 2^-24).
Insertion moves rows and compares: it has to be exact.
"""
import numpy as np
import pytest
import torch

import linear_attention_vlm_b200 as gdn
from oracle import decoding as D

pytestmark = pytest.mark.gpu

DEV = "cuda"


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def tree(rng, n, kind):
    if kind == "star":
        return [-1] * n
    if kind == "chain":
        return list(range(-1, n - 1))
    return [int(rng.integers(max(-1, i - 5), i)) if i else -1 for i in range(n)]


class Case:
    """Inputs of the attention entry points; what no call may use is NaN."""

    def __init__(self, nodes, lens, cap, Hq, Hkv, seed=0, kind="random", q_scale=1.0, pad=0, window=0, ring=False):
        r = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        B, T = len(nodes), sum(nodes)
        bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)  # noqa: E731
        self.B, self.T, self.cap, self.window, self.lens, self.nodes = B, T, cap, window, list(lens), list(nodes)
        self.cu = cu_of(nodes)
        self.q, self.k, self.v = bf(T + pad, Hq, 128) * q_scale, bf(T + pad, Hkv, 128), bf(T + pad, Hkv, 128)
        self.kc, self.vc = bf(B, cap, Hkv, 128), bf(B, cap, Hkv, 128)
        for x in (self.q, self.k, self.v):
            x[T:] = float("nan")
        for b, l in enumerate(lens):
            self.kc[b, l:] = float("nan")
            self.vc[b, l:] = float("nan")
        self.parents = np.array(sum((tree(r, n, kind) for n in nodes), []) + [0] * pad, dtype=np.int64)
        self.pos = self.seen = None
        if ring:
            self.seen = np.array([l + int(r.integers(0, 5000)) for l in lens])
            self.pos = np.zeros((B, Hkv, cap), np.int64)
            for b, l in enumerate(lens):
                for h in range(Hkv):
                    self.pos[b, h, :l] = r.permutation(l) + self.seen[b] - l

    def places(self):
        return {} if self.pos is None else dict(cache_pos=ints(self.pos), seen=ints(self.seen))

    def run(self, chain=False, **kw):
        kw = {**dict(max_nodes=max(self.nodes + [1]), window=self.window), **self.places(), **kw}
        ws = torch.empty(max(16, gdn.gdn_tree_attention_workspace_size(
            self.B, self.q.shape[0], kw["max_nodes"], self.cap, self.q.shape[1], self.k.shape[1])), dtype=torch.uint8, device=DEV)
        o, lse = gdn.gdn_tree_attention(self.q.to(DEV), self.k.to(DEV), self.v.to(DEV), None if chain else ints(self.parents),
                                        self.kc.to(DEV), self.vc.to(DEV), ints(self.lens), ints(self.cu), workspace=ws, **kw)
        assert gdn.gdn_read_status(ws.view(torch.int32)) == 0
        return o, lse

    def ref(self, chain=False, scale=None):
        return D.tree_attention(np64(self.q), np64(self.k), np64(self.v), None if chain else self.parents, np64(self.kc),
                                np64(self.vc), self.lens, self.cu, self.pos, self.seen, self.window, scale)

    def score_error(self, scale=128 ** -0.5):
        big = float(np.nanmax(np.abs(np64(self.q)).sum(-1)) * np.nanmax(np.abs(np.concatenate(
            [np64(self.k).ravel(), np64(self.kc).ravel(), [0.0]]))))
        return 2.0 ** -23 * 128 * scale * big

    def check(self, o, lse, ref, ref_lse, scale=128 ** -0.5):
        T, E = self.T, self.score_error(scale)
        vmax = max(float(np.nanmax(np.abs(np64(self.v)))), float(np.nanmax(np.abs(np64(self.vc)))) if max(self.lens) else 0.0)
        err = np.abs(np64(o)[:T] - ref[:T])
        over = float((err - 2.0 ** -8 * np.abs(ref[:T]) - (2.0 ** -8 + 2 * E) * vmax).max())
        assert over <= 0, "output over its bound by %.3g" % over
        bound = E + (max(self.lens + [0]) / 64 + 64 + 8 + 8 * np.abs(ref_lse[:T])) * 2.0 ** -23
        over = float((np.abs(np64(lse)[:T] - ref_lse[:T]) - bound).max())
        assert over <= 0, "lse over its bound by %.3g" % over


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (4, 4), (3, 1), (5, 5), (24, 2), (1, 1), (40, 1), (128, 1), (200, 2)])
def test_attention_head_layouts(Hq, Hkv):
    # ragged trees and caches: empty ones, lengths around the 128-key block
    nodes, lens = [3, 1, 0, 17, 5, 64], [130, 0, 50, 127, 128, 129]
    c = Case(nodes, lens, 200, Hq, Hkv, seed=Hq)
    c.check(*c.run(), *c.ref())


@pytest.mark.parametrize("kind", ["random", "star", "chain"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 63, 64])
def test_attention_tree_sizes(n, kind):
    c = Case([n, max(1, n // 2)], [300, 65], 300, 16, 2, seed=n, kind=kind)
    c.check(*c.run(), *c.ref())


@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 255, 256, 1000, 5000])
def test_attention_cache_lengths(length):
    # one sequence: many CTAs share it
    c = Case([7], [length], max(1, length + 3), 16, 2, seed=length)
    c.check(*c.run(), *c.ref())


def test_attention_many_short_sequences():
    r = np.random.default_rng(0)
    nodes, lens = [int(x) for x in r.integers(0, 6, 700)], [int(x) for x in r.integers(0, 40, 700)]
    c = Case(nodes, lens, 40, 8, 2, seed=3)
    c.check(*c.run(), *c.ref())


@pytest.mark.parametrize("n", [3, 40])
def test_attention_one_long_sequence_among_short(n):
    c = Case([n, n, 1], [9, 9000, 130], 9001, 16, 2, seed=n)
    c.check(*c.run(), *c.ref())


@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("window", [1, 2, 60, 128, 500])
def test_attention_window(window, ring):
    c = Case([9, 64, 1], [300, 257, 90], 400, 8, 2, seed=window, kind="chain", window=window, ring=ring)
    c.check(*c.run(), *c.ref())
    c = Case([20, 3], [300, 257], 300, 4, 4, seed=window + 1, window=window, ring=ring)
    c.check(*c.run(), *c.ref())


def test_attention_chain_without_parents_and_scale():
    c = Case([20, 64], [100, 40], 128, 8, 4, seed=8, kind="chain")
    a, b = c.run(chain=True), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, lse = c.run(chain=True, scale=0.25)
    c.check(o, lse, *c.ref(chain=True, scale=0.25), scale=0.25)


def test_attention_bad_parents_are_roots():
    c = Case([12, 5], [70, 3], 80, 4, 2, seed=9)
    c.parents[[3, 7, 13, 14]] = [3, 60, -5, 2 ** 30]
    c.check(*c.run(), *c.ref())


@pytest.mark.parametrize("q_scale", [4.0, 12.0])
def test_attention_sharp_scores(q_scale):
    # the running maximum moves from block to block
    c = Case([30, 1], [900, 700], 900, 8, 2, seed=4, q_scale=q_scale)
    c.kc = (c.kc.float() * torch.linspace(0.5, 3.0, 900).view(1, 900, 1, 1)).to(torch.bfloat16)
    c.check(*c.run(), *c.ref())


def test_attention_is_the_window_attention_of_a_run():
    # a prompt's last tokens over the rest as a cache: what gdn_swa_attention gives
    T, cut, Hq, Hkv = 700, 650, 16, 2
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    full = gdn.gdn_swa_attention(q, k, v, window=200)
    o, _ = gdn.gdn_tree_attention(q[cut:], k[cut:], v[cut:], None, k[None, :cut].contiguous(), v[None, :cut].contiguous(),
                                  ints([cut]), window=200)
    # two bf16 results of the same sums: both within the bar of the attention
    assert float((o.float() - full[cut:].float()).abs().max()) <= 2 * (2.0 ** -8 * float(full.abs().max()) + 2.0 ** -8 * float(v.abs().max()))


def test_attention_leaves_rows_behind_the_last_sequence():
    c = Case([5, 0, 9], [64, 10, 200], 200, 16, 2, seed=6, pad=11)
    o = torch.full((c.T + 11, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.T + 11, 16), 7.0, device=DEV)
    c.run(out=o, lse=lse)
    c.check(o, lse, *c.ref())
    assert torch.all(o[c.T:] == 7) and torch.all(lse[c.T:] == 7)


def test_attention_more_nodes_than_said_stay_untouched():
    c = Case([20, 3], [100, 50], 100, 4, 2, seed=2)
    o = torch.full((c.T, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((c.T, 4), 7.0, device=DEV)
    c.run(out=o, lse=lse, max_nodes=16)
    ref, ref_lse = c.ref()
    keep = [t for t in range(c.T) if not 16 <= t < 20]
    assert torch.all(o[16:20] == 7) and torch.all(lse[16:20] == 7)
    assert float(np.abs(np64(o)[keep] - ref[keep]).max()) <= 2.0 ** -8 * 2 * np.nanmax(np.abs(np64(c.v)))


def test_attention_offsets_past_32_bits():
    # the second sequence's slots lie beyond 2^31 elements and 2^32 bytes
    cap, Hkv = 9_000_000, 2
    kc = torch.empty(2, cap, Hkv, 128, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    c = Case([3, 4], [50, 300], 300, 4, Hkv, seed=1)
    for b, l in enumerate(c.lens):
        kc[b, :l], vc[b, :l] = c.kc[b, :l].to(DEV), c.vc[b, :l].to(DEV)
    o, lse = gdn.gdn_tree_attention(c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), ints(c.parents), kc, vc, ints(c.lens), ints(c.cu))
    c.check(o, lse, *c.ref())
    w = torch.zeros(2, Hkv, cap, device=DEV)
    w_out, new = gdn.gdn_cache_weights(c.q.to(DEV), lse, c.k.to(DEV), kc, w, ints(c.lens), ints(c.cu), ints(c.cu))
    ref, ref_new = D.cache_weights(np64(c.q), np64(lse), np64(c.k), np64(c.kc), np.zeros((2, Hkv, 300)), c.lens, c.cu, c.cu)
    assert np.allclose(np64(w_out[:, :, :300]), ref, atol=1e-4) and float(w_out[:, :, 300:].abs().max()) == 0
    args = dict(recent=7, new_weights=new)
    out = gdn.gdn_cache_insert(c.k.to(DEV), c.v.to(DEV), kc, vc, w_out, torch.zeros(2, Hkv, cap, dtype=torch.int32, device=DEV),
                               ints(c.lens), ints(c.lens), ints(c.cu), **args)
    assert torch.equal(kc[1, 300:304], c.k[3:7].to(DEV)) and torch.equal(vc[1, 300:304], c.v[3:7].to(DEV))
    assert out[2].tolist() == [53, 304]


# ---------------------------------------------------------------- attention weights

def check_weights(c, q, lse, cu_q, got, ref, w_in):
    E = c.score_error()
    finite = lse[np.isfinite(lse)]
    size = (float(np.abs(finite).max()) if finite.size else 0.0) + 20
    rows = c.q.shape[1] * c.q.shape[0]
    for g, r, old in zip(got, ref, (w_in, np.zeros_like(ref[1]))):
        g = np64(g)
        assert np.all(np.abs(g - r) <= np.abs(r - old) * (E + 2.0 ** -22 * (8 + size) + rows * 2.0 ** -23) + 2.0 ** -22 * (np.abs(r) + np.abs(old)))


@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (4, 4), (3, 1), (40, 1), (200, 2)])
@pytest.mark.parametrize("window,ring", [(0, False), (40, False), (40, True), (150, True)])
def test_weights(Hq, Hkv, window, ring):
    c = Case([6, 0, 17, 3, 40], [130, 20, 0, 257, 128], 260, Hq, Hkv, seed=Hq + window, kind="chain", window=window, ring=ring)
    _, lse = c.run()
    lse[2, 0] = float("-inf")                           # an empty row adds nothing
    take = [2, 0, 17, 1, 33]                            # the last queries of every sequence
    rows = np.concatenate([np.arange(c.cu[b + 1] - n, c.cu[b + 1]) for b, n in enumerate(take)])
    q, l, cu_q = c.q[rows], lse[rows], cu_of(take)
    w = torch.rand(c.B, Hkv, c.cap)
    for b, n in enumerate(c.lens):
        w[b, :, n:] = float("nan")
    wd = w.to(DEV)
    got = gdn.gdn_cache_weights(q.to(DEV), l, c.k.to(DEV), c.kc.to(DEV), wd, ints(c.lens), ints(cu_q), ints(c.cu), window=window,
                                weights_out=torch.full_like(wd, 7.0), **c.places())
    ref = D.cache_weights(np64(q), np64(l), np64(c.k), np64(c.kc), np64(w), c.lens, cu_q, c.cu, c.pos, c.seen, window)
    for b, n in enumerate(c.lens):                      # what lies behind the length stays
        assert torch.all(got[0][b, :, n:] == 7)
        got[0][b, :, n:], ref[0][b, :, n:], w[b, :, n:] = 0, 0, 0
    check_weights(c, q, np64(l), cu_q, got, ref, np64(w))
    again = gdn.gdn_cache_weights(q.to(DEV), l, c.k.to(DEV), c.kc.to(DEV), wd, ints(c.lens), ints(cu_q), ints(c.cu), window=window,
                                  **c.places())
    assert again[0] is wd                               # in place, and the same bits
    for b, n in enumerate(c.lens):
        assert torch.equal(again[0][b, :, :n], got[0][b, :, :n])
    assert torch.equal(again[1], got[1])


def test_weights_of_a_whole_prompt_and_uniform_sequences():
    c = Case([64, 64], [0, 0], 1, 8, 2, seed=5, kind="chain")
    _, lse = c.run()
    got = gdn.gdn_cache_weights(c.q.to(DEV), lse, c.k.to(DEV), c.kc.to(DEV), torch.zeros(2, 2, 1, device=DEV), ints(c.lens))
    ref = D.cache_weights(np64(c.q), np64(lse), np64(c.k), np64(c.kc), np.zeros((2, 2, 1)), c.lens, c.cu, c.cu)
    check_weights(c, c.q, np64(lse), c.cu, got, ref, np.zeros((2, 2, 1)))
    assert abs(float(got[1].sum()) - 2 * 64 * 8) <= 1e-3 * 1024      # every query's weights add up to one


def test_weights_of_a_long_prompt():
    # 300 queries of 700 tokens: several blocks of both, causal between them
    T, nq, Hq, Hkv = 700, 300, 6, 2
    gen = torch.Generator().manual_seed(3)
    c = Case([T], [0], 1, Hq, Hkv, seed=6, kind="chain")
    q = c.q[T - nq:]
    lse = torch.randn(nq, Hq, generator=gen) + 7
    got = gdn.gdn_cache_weights(q.to(DEV), lse.to(DEV), c.k.to(DEV), c.kc.to(DEV), torch.zeros(1, Hkv, 1, device=DEV), ints([0]),
                                ints([0, nq]), ints([0, T]))
    ref = D.cache_weights(np64(q), np64(lse), np64(c.k), np64(c.kc), np.zeros((1, Hkv, 1)), [0], [0, nq], [0, T])
    check_weights(c, q, np64(lse), None, got, ref, np.zeros((1, Hkv, 1)))


def test_weights_without_queries_or_tokens():
    c = Case([3, 2], [40, 0], 50, 4, 2, seed=1)
    w = torch.rand(2, 2, 50, device=DEV)
    got = gdn.gdn_cache_weights(c.q[:0].to(DEV), torch.zeros(0, 4, device=DEV), c.k.to(DEV), c.kc.to(DEV), w, ints(c.lens),
                                ints([0, 0, 0]), ints(c.cu), weights_out=torch.zeros_like(w))
    assert torch.equal(got[0][0, :, :40], w[0, :, :40]) and float(got[1].abs().max()) == 0
    got = gdn.gdn_cache_weights(c.q[:0].to(DEV), torch.zeros(0, 4, device=DEV), c.k[:0].to(DEV), c.kc.to(DEV), w.clone(),
                                ints(c.lens))
    assert torch.equal(got[0], w)


# ---------------------------------------------------------------- the tree step

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,kind", [([1], "chain"), ([7, 0, 1, 16], "random"), ([17, 32, 5], "random"), ([33, 64, 2], "random"),
                                        ([64, 40], "chain"), ([50], "star")])
def test_step(dtype, d, nodes, kind):
    r = np.random.default_rng(d + sum(nodes))
    H, T, B = 3, sum(nodes), len(nodes)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    t = lambda x: torch.tensor(x, dtype=torch.float32).to(dtype)    # noqa: E731
    q, k, v = t(unit(r.standard_normal((T, H, d)))), t(unit(r.standard_normal((T, H, d)))), t(r.standard_normal((T, H, d)))
    g = torch.tensor(-0.3 * np.abs(r.standard_normal((T, H))), dtype=torch.float32)
    beta = torch.rand(T, H, generator=torch.Generator().manual_seed(T))
    S = torch.tensor(0.3 * r.standard_normal((B, H, d, d)), dtype=torch.float32)
    parents = np.array(sum((tree(r, n, kind) for n in nodes), []), dtype=np.int64)
    pad = 2
    grow = lambda x: torch.cat([x, torch.full((pad,) + x.shape[1:], float("nan"), dtype=x.dtype)]).to(DEV)  # noqa: E731
    out = torch.full((T + pad, H, d), 7.0, dtype=dtype, device=DEV)
    Sd = S.to(DEV)
    gdn.gdn_tree_step(grow(q), grow(k), grow(v), grow(g), grow(beta), ints(list(parents) + [0] * pad), Sd, ints(cu_of(nodes)),
                      max_nodes=max(nodes), out=out)
    ref = D.tree_step(np64(q), np64(k), np64(v), np64(g), np64(beta), parents, np64(S), cu_of(nodes))
    err = np.abs(np64(out)[:T] - ref)
    if dtype == torch.float32:
        assert float(err.max()) <= 1e-4 * float(np.abs(ref).max())
    else:
        size = max(float(np.linalg.norm(np64(S), axis=-1).max()), float(np.abs(np64(v)).max()))
        assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 7e-4 * size), float(err.max())
    assert torch.all(out[T:] == 7) and torch.equal(Sd.cpu(), S)
    if kind == "chain":
        a = gdn.gdn_tree_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), None, Sd, ints(cu_of(nodes)))
        assert torch.equal(a, out[:T])


@pytest.mark.parametrize("d,nodes", [(64, 33), (128, 1), (128, 16), (128, 64)])
def test_step_in_fp32_is_as_exact_as_fp32(d, nodes):
    """In the norm: operands are off by 2^-21 at most, with either sign (2^-22 in
    the mean of their squares, two of them 2^-21.5), one of four partial products
    is left out (2^-22), sums are rounded d/16 + n/8 times by half a step, with
    either sign (under 2^-22): below 2^-20."""
    gen = torch.Generator().manual_seed(nodes)
    mk = lambda *s: torch.randn(s, generator=gen)                                # noqa: E731
    B, H = 4, 3
    T = B * nodes
    q, k = (torch.nn.functional.normalize(mk(T, H, d), dim=-1) for _ in range(2))
    v, g, beta, S = mk(T, H, d), -0.2 * mk(T, H).abs(), torch.rand(T, H, generator=gen), mk(B, H, d, d)
    parents, cu = [i // 2 - 1 for _ in range(B) for i in range(nodes)], cu_of([nodes] * B)
    out = gdn.gdn_tree_step(*(x.to(DEV) for x in (q, k, v, g, beta)), ints(parents), S.to(DEV), ints(cu))
    ref = D.tree_step(*(np64(x) for x in (q, k, v, g, beta)), parents, np64(S), cu)
    assert np.linalg.norm(np64(out) - ref) <= 2.0 ** -20 * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("what", [0, 1, 2])
def test_step_does_not_hide_a_nan(dtype, what):
    """A NaN of arithmetic on the device (all bits of its fraction set) in q, k
    or v reaches the output of its node; other sequences stay as they are."""
    gen = torch.Generator().manual_seed(what)
    t = [(0.1 * torch.randn(6, 2, 128, generator=gen)).to(dtype).to(DEV) for _ in range(3)]
    g, beta = -torch.rand(6, 2, generator=gen).to(DEV), torch.full((6, 2), 0.5, device=DEV)
    S = torch.randn(2, 2, 128, 128, generator=gen).to(DEV)
    clean = gdn.gdn_tree_step(*t, g, beta, None, S, ints([0, 3, 6]))
    zero = torch.zeros(1, device=DEV)
    t[what][1, 0, 5:6] = (zero / zero).to(dtype)
    out = gdn.gdn_tree_step(*t, g, beta, None, S, ints([0, 3, 6]))
    assert bool(out[1, 0].isnan().any())
    assert torch.equal(out[3:], clean[3:]) and torch.equal(out[:, 1], clean[:, 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_of_a_root_is_a_decode_step(dtype):
    B, H, d = 5, 4, 128
    gen = torch.Generator().manual_seed(0)
    x = lambda *s: torch.randn(s, generator=gen)                                 # noqa: E731
    q, k, v = (torch.nn.functional.normalize(x(B, H, d), dim=-1).to(dtype).to(DEV) for _ in range(3))
    g, beta, S = (-0.1 * x(B, H).abs()).to(DEV), torch.sigmoid(x(B, H)).to(DEV), x(B, H, d, d).to(DEV)
    got = gdn.gdn_tree_step(q, k, v, g, beta, None, S)
    ref, _ = gdn.gdn_decode_step(q, k, v, g, beta, S.clone())
    tol = 1e-4 if dtype == torch.float32 else 2.0 ** -7
    assert float((got.float() - ref.float()).abs().max()) <= tol * float(ref.float().abs().max())


def test_step_strong_decay_and_full_writes():
    # exp(g) far below the fp32 range along a path, beta of 0 and 1
    n, H, d = 40, 2, 128
    gen = torch.Generator().manual_seed(4)
    x = lambda *s: torch.randn(s, generator=gen)                                 # noqa: E731
    q, k = (torch.nn.functional.normalize(x(n, H, d), dim=-1).to(torch.bfloat16) for _ in range(2))
    v, S = x(n, H, d).to(torch.bfloat16), x(1, H, d, d)
    g = -20 * torch.rand(n, H, generator=gen)
    beta = (torch.rand(n, H, generator=gen) > 0.5).float()
    out = gdn.gdn_tree_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), beta.to(DEV), None, S.to(DEV))
    ref = D.tree_step(np64(q), np64(k), np64(v), np64(g), np64(beta), None, np64(S), [0, n])
    assert np.all(np.abs(np64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 7e-4 * float(np.linalg.norm(np64(S), axis=-1).max()))


# ---------------------------------------------------------------- insertion

def run_insert(lens, ms, cap, Hkv, recent, seed, dtype=torch.bfloat16, d=128, weights=None, new=True, in_place=True, far=0):
    r = np.random.default_rng(seed)
    B, T = len(lens), sum(ms)
    gen = torch.Generator().manual_seed(seed)
    k, v = torch.randn(T, Hkv, d, generator=gen).to(dtype), torch.randn(T, Hkv, d, generator=gen).to(dtype)
    kc, vc = torch.randn(B, cap, Hkv, d, generator=gen).to(dtype), torch.randn(B, cap, Hkv, d, generator=gen).to(dtype)
    w = weights(r, (B, Hkv, cap)) if weights else np.maximum(r.standard_normal((B, Hkv, cap)), 0).astype(np.float32)
    nw = (weights(r, (T, Hkv)) if weights else np.maximum(r.standard_normal((T, Hkv)), 0).astype(np.float32)) if new else None
    seen = np.array([l + far for l in lens])
    pos = np.zeros((B, Hkv, cap), np.int64)
    for b, l in enumerate(lens):
        for h in range(Hkv):
            pos[b, h, :l] = r.permutation(l) + far
    cu = cu_of(ms)
    ref = D.cache_insert(w, pos, lens, seen, cu, recent, cap, nw)
    D_ = lambda x, dt: torch.tensor(np.asarray(x), dtype=dt, device=DEV)  # noqa: E731
    wi, pi, li, si = D_(w, torch.float32), D_(pos, torch.int32), D_(lens, torch.int32), D_(seen, torch.int32)
    outs = {} if in_place else dict(weights_out=wi.clone(), pos_out=pi.clone(), lens_out=torch.zeros_like(li), seen_out=torch.zeros_like(si))
    kd, vd = kc.to(DEV), vc.to(DEV)
    got = gdn.gdn_cache_insert(k.to(DEV), v.to(DEV), kd, vd, wi, pi, li, si, D_(cu, torch.int32), recent=recent,
                               new_weights=None if nw is None else D_(nw, torch.float32), **outs)
    gw, gp, gl, gs, slots = (x.cpu().numpy() for x in got)
    assert gl.tolist() == ref[2].tolist() and gs.tolist() == ref[3].tolist()
    assert np.array_equal(slots, ref[4])
    for b in range(B):
        n = ref[2][b]
        assert np.array_equal(gp[b, :, :n], ref[1][b, :, :n])
        assert np.array_equal(gw[b, :, :n], ref[0][b, :, :n].astype(np.float32), equal_nan=True)
        for j in range(cu[b], cu[b + 1]):
            for h in range(Hkv):
                if ref[4][j, h] >= 0:
                    kc[b, ref[4][j, h], h], vc[b, ref[4][j, h], h] = k[j, h], v[j, h]
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("recent", [0, 7, 100, 300])
def test_insert_ragged(recent, in_place):
    # room left, exactly full, more tokens than slots, nothing new, nothing cached
    run_insert([300, 290, 0, 300, 10, 300, 0], [4, 15, 500, 0, 290, 299, 0], 300, 2, recent, recent, in_place=in_place)


@pytest.mark.parametrize("cap,ms,recent", [(1, [1, 3], 0), (1, [2], 1), (33, [1], 5), (1024, [1, 1024, 1025], 0), (5000, [300, 7000], 64),
                                           (40000, [70000], 1000)])
def test_insert_sizes(cap, ms, recent):
    run_insert([cap if i % 2 == 0 and cap < 40000 else 0 for i in range(len(ms))], ms, cap, 1, recent, cap + recent, d=64)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 4), (torch.float32, 128), (torch.bfloat16, 8), (torch.bfloat16, 576)])
def test_insert_row_sizes(dtype, d):
    run_insert([50, 20], [9, 70], 50, 3, 5, d, dtype=dtype, d=d)


@pytest.mark.parametrize("Hkv", [5, 7, 8, 9, 16])
@pytest.mark.parametrize("ms,in_place", [([1, 0, 9], True), ([200, 3, 1], False), ([6] * 40, True)])
def test_insert_heads_and_lists(Hkv, ms, in_place):
    # few rows a head, many rows a head, more lists than SMs
    run_insert([100 - i % 3 for i in range(len(ms))], ms, 100, Hkv, 20, Hkv, d=64, in_place=in_place)


def test_insert_many_rows_of_many_lists():
    run_insert([70] * 75, [30 + 5 * (i % 9) for i in range(75)], 70, 1, 10, 4)


def odd_weights(r, shape):
    """Many ties, zeros of both signs, negatives, infinities and NaN."""
    return r.choice(np.array([0.0, -0.0, 1.0, 1.0, -2.0, np.inf, -np.inf, np.nan, 1e-40, 3e38], np.float32), shape)


@pytest.mark.parametrize("recent", [0, 20])
def test_insert_odd_weights_and_ties(recent):
    run_insert([200, 200, 13], [30, 250, 400], 200, 2, recent, 5, weights=odd_weights)
    run_insert([200], [90], 200, 2, recent, 6, weights=lambda r, s: np.zeros(s, np.float32))


def test_insert_without_new_weights_far_into_a_stream():
    run_insert([100, 40], [10, 100], 100, 2, 30, 3, new=False, far=2_000_000_000)


# ---------------------------------------------------------------- streams, graphs, and the operators together

def test_on_another_stream_and_captured():
    c = Case([9, 30], [700, 200], 800, 16, 2, seed=2)
    q, k, v, kc, vc = (x.to(DEV) for x in (c.q, c.k, c.v, c.kc, c.vc))
    lens, cu, parents = ints(c.lens), ints(c.cu), ints(c.parents)
    ws = [torch.empty(gdn.gdn_tree_attention_workspace_size(2, c.T, 30, 800, 16, 2), dtype=torch.uint8, device=DEV) for _ in range(2)]
    w = torch.zeros(2, 2, 800, device=DEV)
    outs = [(torch.zeros_like(q), torch.zeros(c.T, 16, device=DEV)) for _ in range(2)]
    ww = torch.empty(gdn.gdn_cache_weights_workspace_size(2, c.T, c.T, 800, 16, 2), dtype=torch.uint8, device=DEV)

    def step(i):
        gdn.gdn_tree_attention(q, k, v, parents, kc, vc, lens, cu, max_nodes=30, out=outs[i][0], lse=outs[i][1], workspace=ws[i])
        return gdn.gdn_cache_weights(q, outs[i][1], k, kc, w, lens, cu, cu, weights_out=torch.empty_like(w), workspace=ww)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0)
    torch.cuda.current_stream().wait_stream(side)
    c.check(*outs[0], *c.ref())
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    got = []
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            got.append(step(i))
    # the lengths are read when the graph runs, not when it is captured
    c.lens = [133, 199]
    lens.copy_(ints(c.lens))
    for o, l in outs:
        o.zero_(), l.zero_()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    ref = c.ref()
    for o, l in outs:
        c.check(o, l, *ref)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(got[0][1], got[1][1])


def test_a_stream_of_drafts():
    """Speculative decoding of one hybrid block over a bounded cache: drafts
    are verified by both mixers, a path is accepted, its attention weights are
    added up, its tokens enter the cache and the state.  Every step is checked
    against the oracle on the same cache."""
    r = np.random.default_rng(0)
    gen = torch.Generator().manual_seed(0)
    B, cap, Hq, Hkv, H, recent = 3, 48, 8, 2, 2, 16
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)             # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(s, generator=gen), dim=-1).to(torch.bfloat16)  # noqa: E731
    kc, vc = torch.full((B, cap, Hkv, 128), float("nan"), dtype=torch.bfloat16, device=DEV), None
    vc = kc.clone()
    w = torch.zeros(B, Hkv, cap, device=DEV)
    pos = torch.zeros(B, Hkv, cap, dtype=torch.int32, device=DEV)
    lens, seen = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    S = torch.zeros(B, H, 128, 128, device=DEV)
    S_ref = np.zeros((B, H, 128, 128))
    import oracle
    for turn in range(30):
        nodes = [int(x) for x in r.integers(1, 14, B)]
        T, cu = sum(nodes), cu_of(nodes)
        parents = sum((tree(r, n, "random") for n in nodes), [])
        q, k, v = bf(T, Hq, 128), bf(T, Hkv, 128), bf(T, Hkv, 128)
        c = Case(nodes, lens.tolist(), cap, Hq, Hkv, window=40)
        c.q, c.k, c.v, c.kc, c.vc, c.parents = q, k, v, kc.cpu(), vc.cpu(), np.array(parents)
        c.pos, c.seen = pos.cpu().numpy(), seen.cpu().numpy()
        o, lse = gdn.gdn_tree_attention(q.to(DEV), k.to(DEV), v.to(DEV), ints(parents), kc, vc, lens, ints(cu), cache_pos=pos,
                                        seen=seen, window=40)
        c.check(o, lse, *c.ref())
        gq, gk, gv = unit(T, H, 128), unit(T, H, 128), bf(T, H, 128)
        g, beta = -0.1 * torch.rand(T, H, generator=gen), torch.rand(T, H, generator=gen)
        out = gdn.gdn_tree_step(gq.to(DEV), gk.to(DEV), gv.to(DEV), g.to(DEV), beta.to(DEV), ints(parents), S, ints(cu))
        ref = D.tree_step(np64(gq), np64(gk), np64(gv), np64(g), np64(beta), parents, np64(S), cu)
        size = max(float(np.linalg.norm(np64(S), axis=-1).max()), float(np.abs(np64(gv)).max()))
        assert np.all(np.abs(np64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 7e-4 * size)
        # accept one line of every tree
        lines = [D.paths(parents[cu[b]:cu[b + 1]], n)[int(r.integers(0, n))] for b, n in enumerate(nodes)]
        rows = torch.tensor([int(cu[b]) + i for b, line in enumerate(lines) for i in line])
        cua = cu_of([len(x) for x in lines])
        before = [x.cpu().numpy() for x in (w, pos, lens, seen)]
        w, new = gdn.gdn_cache_weights(q[rows].to(DEV), lse[rows.to(DEV)], k[rows].to(DEV), kc, w, lens, ints(cua), ints(cua),
                                       cache_pos=pos, seen=seen, window=40)
        ref_w = D.cache_weights(np64(q[rows]), np64(lse)[rows], np64(k[rows]), np64(kc), before[0], before[2], cua, cua, before[1],
                                before[3], 40)
        for b, n in enumerate(before[2]):
            assert np.allclose(np64(w)[b, :, :n], ref_w[0][b, :, :n], rtol=1e-4, atol=1e-5)
        assert np.allclose(np64(new), ref_w[1], rtol=1e-4, atol=1e-5)
        ref_i = D.cache_insert(w.cpu().numpy(), before[1], before[2], before[3], cua, recent, cap, new.cpu().numpy())
        w, pos, lens, seen, slots = gdn.gdn_cache_insert(k[rows].to(DEV), v[rows].to(DEV), kc, vc, w, pos, lens, seen, ints(cua),
                                                         recent=recent, new_weights=new)
        assert np.array_equal(slots.cpu().numpy(), ref_i[4]) and lens.tolist() == ref_i[2].tolist()
        for b, n in enumerate(ref_i[2]):
            assert np.array_equal(pos.cpu().numpy()[b, :, :n], ref_i[1][b, :, :n])
        _, S = gdn.gdn_prefill(*(x[rows].to(DEV) for x in (gq, gk, gv, g, beta)), S, ints(cua))
        _, S_ref = oracle.prefill(*(np64(x[rows]) for x in (gq, gk, gv, g, beta)), S_ref, cua)
        assert np.abs(np64(S) - S_ref).max() <= 2e-2 * np.abs(S_ref).max()
    assert lens.tolist() == [cap] * B
