"""Bars of the attention over a cache and of the bf16 tree step that a lost
slot, a lost block or a lost half of an operand oversteps.

On the CPU the bars are tried on restatements of the operators with the kernels'
roundings: the right ones pass, ones with a slot or a block left out, a half
block of V taken for another or the low halves of an operand dropped do not.
On the GPU (marked) the kernels are held to the same bars.

Attention, every element:
  |o - ref| <= 2^-8 |ref| + (2^-8 + 2 E + 2^-16) sum_s p_s |v_s|
the rounding of o, of every p_s, and what an error E of the scores and the fp32 sums (at most
64 + L / 64 + 8 additions of 2^-24 each, below 2^-16 for L <= 10000) make of the mean;
  |lse - ref| <= E + (L / 64 + 64 + 8 + 8 |ref|) 2^-23,
E = 2^-23 d scale max_s sum_i |q_i k_si| per row (d additions, cut at worst).
V is positive, one channel per slot, so that a channel is a mean over L / 128
slots: of up to 9000, one lost costs it 1.3 % or more, against a bar of 0.8 %.
Attention with V of normal numbers, in the norm: roundings of a half step at
most, uniform in it, are off by 2^-8 / sqrt(3) in the root mean square at the
foot of a binade and by less above, and are independent, so
  ||o - ref||^2 <= (2^-16 / 3) (||ref||^2 + sum p_s^2 v_s^2) (1 + 1/10),
a tenth for the sample (thousands of elements) and E.

Tree step in bf16: an output is the bf16 of the result plus a small error e, so
it differs from the bf16 of the exact result by |e| in the mean (the step
between two bf16 numbers, as often as e crosses their middle):
  mean |out - bf16(ref)| <= mean e,
  e = 2^-16 gamma |S||q| + 3 2^-16 |M| (beta (|v| + gamma |S||k|)),
where S, R and M are off by 2^-17 each (R also by what S is off), the product of the low
halves of M and R is left out (2^-16) and fp32 sums of 64 to 192 terms, 16 at a
time in the tensor core, are off by 2^-18.
"""
import math

import numpy as np
import pytest
import torch

from oracle import decoding as D

SCALE = 128 ** -0.5


def bf16(x):
    """Rounded to bf16, in fp64."""
    return torch.as_tensor(x).to(torch.bfloat16).double()


# ---------------------------------------------------------------- attention

class Rows:
    """One (sequence, key/value head): rows [R, 128], keys and values [S, 128]
    of the slots and then the nodes, and which of them a row sees."""

    def __init__(self, q, keys, vals, sees):
        x = (q @ keys.T * SCALE).masked_fill(~sees, -math.inf)
        self.p = torch.softmax(x, -1)
        self.lse = torch.logsumexp(x, -1)
        self.o = self.p @ vals
        self.size = self.p @ vals.abs()
        self.square = (self.p ** 2) @ (vals ** 2)
        self.E = (2.0 ** -23 * 128 * SCALE * (q.abs() @ keys.abs().T)).masked_fill(~sees, 0).amax(-1)
        self.L, self.vals, self.x = keys.shape[0], vals, x

    def rounded(self, vals=None, sees=None):
        """The result with the kernel's roundings; ``sees``: slots left in."""
        x = self.x if sees is None else self.x.masked_fill(~sees, -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        o = bf16(p) @ (self.vals if vals is None else vals) / p.sum(-1, keepdim=True)
        return bf16(o), torch.logsumexp(x, -1)

    def within_elements(self, o, lse):
        bar = 2.0 ** -8 * self.o.abs() + (2.0 ** -8 + 2 * self.E[:, None] + 2.0 ** -16) * self.size
        bar_lse = self.E + (self.L / 64 + 64 + 8 + 8 * self.lse.abs()) * 2.0 ** -23
        return bool(((o - self.o).abs() <= bar).all()), bool(((lse - self.lse).abs() <= bar_lse).all())

    def within_norm(self, o):
        return float((o - self.o).square().sum()) <= 2.0 ** -16 / 3 * 1.1 * float(self.o.square().sum() + self.square.sum())


CASES = [   # nodes, lengths: items cut over all CTAs, by keys and by rows; one long among short; full and ragged blocks
    ([7], [5000]), ([40], [5000]), ([3, 3, 1], [9, 9000, 130]), ([40, 40, 1], [9, 9000, 130]), ([1], [8192]), ([64], [300]),
]
HQ, HKV = 16, 2


class Batch:
    def __init__(self, nodes, lens, every_slot, seed=0):
        r = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        T, B, cap = sum(nodes), len(nodes), max(lens) + 5
        mk = lambda *s: torch.randn(s, generator=gen)                            # noqa: E731
        self.nodes, self.lens = nodes, lens
        self.cu = np.concatenate([[0], np.cumsum(nodes)])
        self.parents = [int(r.integers(max(-1, i - 5), i)) if i else -1 for n in nodes for i in range(n)]
        # nearly even probabilities where every slot is to count
        self.q = (mk(T, HQ, 128) * (0.05 if every_slot else 1.0)).to(torch.bfloat16)
        self.k, self.kc = mk(T, HKV, 128).to(torch.bfloat16), mk(B, cap, HKV, 128).to(torch.bfloat16)
        if every_slot:
            def one_channel(n):
                v = torch.zeros(n, HKV, 128)
                s = torch.arange(n)
                for h in range(HKV):
                    v[s, h, (s * 37 + s // 128 * 11 + h) % 128] = 1 + torch.rand(n, generator=gen) / 8
                return v
            self.v = one_channel(T).to(torch.bfloat16)
            self.vc = torch.stack([one_channel(cap) for _ in range(B)]).to(torch.bfloat16)
        else:
            self.v, self.vc = mk(T, HKV, 128).to(torch.bfloat16), mk(B, cap, HKV, 128).to(torch.bfloat16)

    def heads(self):
        """(rows of the packed result, first query head, Rows) of every sequence and head."""
        g = HQ // HKV
        for b, (n, l) in enumerate(zip(self.nodes, self.lens)):
            t = slice(int(self.cu[b]), int(self.cu[b + 1]))
            sees = torch.zeros(n, l + n, dtype=torch.bool)
            sees[:, :l] = True
            for i, line in enumerate(D.paths(self.parents[t], n)):
                sees[i, [l + j for j in line]] = True
            for h in range(HKV):
                keys = torch.cat([self.kc[b, :l, h], self.k[t, h]]).double()
                vals = torch.cat([self.vc[b, :l, h], self.v[t, h]]).double()
                q = self.q[t, h * g:(h + 1) * g].double().reshape(n * g, 128)
                yield t, h * g, Rows(q, keys, vals, sees.repeat_interleave(g, 0))


def verdicts(b, o, lse, what):
    g = HQ // HKV
    for t, h, rows in b.heads():
        oo, ll = o[t, h:h + g].reshape(-1, 128), lse[t, h:h + g].reshape(-1)
        yield rows.within_elements(oo, ll) if what else rows.within_norm(oo)


@pytest.mark.parametrize("nodes,lens", [c for c in CASES if max(c[1]) > 1000], ids=str)
def test_bars_of_the_attention_see_a_lost_slot_and_a_lost_block(nodes, lens):
    b, normal = Batch(nodes, lens, True), Batch(nodes, lens, False)
    at = HKV * int(np.argmax(lens))
    (_, _, rows), (_, _, plain) = list(b.heads())[at], list(normal.heads())[at]
    l = max(lens)
    assert all(rows.within_elements(*rows.rounded())) and plain.within_norm(plain.rounded()[0])
    for lost in (0, 127, 128, 4000, l - 1):
        keep = torch.ones(rows.x.shape, dtype=torch.bool)
        keep[:, lost] = False
        assert rows.within_elements(*rows.rounded(sees=keep)) == (False, False), lost
        vals = rows.vals.clone()
        vals[lost] = 0                                       # in the product with V alone
        assert not rows.within_elements(*rows.rounded(vals=vals))[0], lost
    for block in (0, 128 * 20, l // 128 * 128 - 128):
        vals = plain.vals.clone()
        vals[block:block + 128] = 0
        assert not plain.within_norm(plain.rounded(vals=vals)[0]), block
        vals = plain.vals.clone()
        vals[[*range(block, block + 64)]] = plain.vals[block + 64:block + 128]   # one half in place of the other
        assert not plain.within_norm(plain.rounded(vals=vals)[0]), block


@pytest.mark.gpu
@pytest.mark.parametrize("every_slot", [True, False])
@pytest.mark.parametrize("nodes,lens", CASES, ids=str)
def test_attention_counts_every_slot_and_block(nodes, lens, every_slot):
    import linear_attention_vlm_b200 as gdn
    b = Batch(nodes, lens, every_slot, seed=len(nodes) + max(nodes))
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()       # noqa: E731
    o, lse = gdn.gdn_tree_attention(b.q.cuda(), b.k.cuda(), b.v.cuda(), ints(b.parents), b.kc.cuda(), b.vc.cuda(),
                                    ints(b.lens), ints(b.cu), max_nodes=max(nodes))
    got = list(verdicts(b, o.cpu().double(), lse.cpu().double(), every_slot))
    assert all(got) if not every_slot else all(x and y for x, y in got), got


# ---------------------------------------------------------------- the tree step in bf16

STEPS = [(64, 16, "random"), (64, 64, "chain"), (128, 7, "random"), (128, 32, "random"), (128, 64, "random"), (128, 64, "chain")]


class Step:
    """Inputs of one sequence of H heads and the closed form of their result."""

    def __init__(self, d, n, kind, H=4, seed=0):
        r = np.random.default_rng(seed + d + n)
        mk = lambda *s: torch.tensor(r.standard_normal(s))                       # noqa: E731
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)                        # noqa: E731
        self.n, self.H, self.d = n, H, d
        self.q, self.k, self.v = (x.to(torch.bfloat16) for x in (unit(mk(n, H, d)), unit(mk(n, H, d)), mk(n, H, d)))
        self.g, self.beta = (-0.3 * mk(n, H).abs()).float(), torch.tensor(r.random((n, H)), dtype=torch.float32)
        self.S = mk(1, H, d, d).float()
        self.parents = list(range(-1, n - 1)) if kind == "chain" else [int(r.integers(max(-1, i - 5), i)) if i else -1 for i in range(n)]
        anc = torch.zeros(n, n, dtype=torch.bool)
        for i, line in enumerate(D.paths(self.parents, n)):
            anc[i, line] = True
        h = lambda x: x.double().transpose(0, 1)                                 # noqa: E731  [H, n, ...]
        q, k, self.v64, self.b = h(self.q), h(self.k), h(self.v), h(self.beta)[..., None]
        G = h(self.g) @ anc.double().T
        decay = torch.where(anc, torch.where(anc, G[:, :, None] - G[:, None, :], torch.zeros(())).exp(), torch.zeros((), dtype=torch.float64))
        self.gamma = G.exp()[..., None]
        A = self.b * decay * (k @ k.transpose(1, 2)) * (1 - torch.eye(n))
        P = decay * (q @ k.transpose(1, 2))
        self.M = torch.linalg.solve(torch.eye(n, dtype=torch.float64) + A, P, left=False)
        self.q64, self.k64, self.S64 = q, k, self.S[0].double()
        self.ref = self.result()
        ab = lambda x: x.abs()                                                   # noqa: E731
        St = ab(self.S64).transpose(1, 2)
        reach = self.b * (ab(self.v64) + self.gamma * (ab(k) @ St))
        self.e = float((2.0 ** -16 * self.gamma * (ab(q) @ St) + 3 * 2.0 ** -16 * (ab(self.M) @ reach)).mean())

    def result(self, S=None, round_r=lambda x: x, round_m=lambda x: x):
        S = self.S64 if S is None else S
        R = self.b * (self.v64 - self.gamma * (self.k64 @ S.transpose(1, 2)))
        return self.gamma * (self.q64 @ S.transpose(1, 2)) + round_m(self.M) @ round_r(R)

    def within(self, out):
        return float((out - bf16(self.ref)).abs().mean()) <= self.e


def pair(x):
    """As a pair of bf16 numbers."""
    hi = bf16(x.float())
    return hi + bf16((x - hi).float())


@pytest.mark.parametrize("d,n,kind", STEPS)
def test_bar_of_the_step_sees_a_lost_low_half(d, n, kind):
    s = Step(d, n, kind)
    t = [x.double().numpy() for x in (s.q, s.k, s.v, s.g, s.beta)]
    assert np.allclose(D.tree_step(*t, s.parents, s.S.double().numpy(), [0, n]).transpose(1, 0, 2), s.ref.numpy(), atol=1e-10)
    assert s.within(bf16(s.result(pair(s.S64), pair, pair)))
    assert not s.within(bf16(s.result(bf16(s.S64), pair, pair)))
    assert not s.within(bf16(s.result(pair(s.S64), bf16, pair)))
    if n > 7:   # few nodes see little of one another: at 7, what M loses is below what S may lose
        assert not s.within(bf16(s.result(pair(s.S64), pair, bf16)))


@pytest.mark.gpu
@pytest.mark.parametrize("d,n,kind", STEPS)
def test_step_in_bf16_keeps_the_low_halves(d, n, kind):
    import linear_attention_vlm_b200 as gdn
    s = Step(d, n, kind, seed=1)
    out = gdn.gdn_tree_step(*(x.cuda() for x in (s.q, s.k, s.v, s.g, s.beta)),
                            torch.tensor(s.parents, dtype=torch.int32).cuda(), s.S.cuda())
    out = out.cpu().double().transpose(0, 1)
    assert s.within(out), (float((out - bf16(s.ref)).abs().mean()), s.e)
