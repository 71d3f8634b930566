"""The tree step under strong gates: a node whose gate closes almost wholly
leaves the nodes below it as exact as any other.

Bars, in the norm of every sequence and head.  fp32: 2^-20 for products and sums (operands
off by 2^-21 with either sign, one of four partial products left out, sums
rounded); the decays of a path add next to nothing as long as its sum of gates
is kept to more bits than fp32 has: the exponent of a pair D apart is rounded
to 2^-24 D, which weighs exp(-D) D 2^-24 < 2^-25, and its own error (2^-43 of
the path sum, here at most 2^20) is below 2^-23.  bf16: the rounding of the output, a half
step at most, uniform in it: 2^-8 / sqrt(3) at the foot of a binade and less
above.
"""
import numpy as np
import pytest
import torch

import linear_attention_vlm_b200 as gdn
from oracle import decoding as D

pytestmark = pytest.mark.gpu

DEV = "cuda"


def gates(rng, n, kind, strong):
    g = -0.05 * np.abs(rng.standard_normal(n))
    if kind == "root":
        g[0] = strong
    elif kind == "middle":
        g[n // 4] = strong
    else:
        g[::8] = strong
    return g.astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,nodes", [(64, 16), (64, 33), (128, 32), (128, 64)])
@pytest.mark.parametrize("kind,strong", [("root", -75.0), ("middle", -20.0), ("middle", -50.0), ("many", -20.0), ("middle", -1e4),
                                         ("root", -1e6), ("many", -1e5)])
def test_nodes_below_a_strong_gate(dtype, d, nodes, kind, strong):
    r = np.random.default_rng(nodes + d)
    H, B = 2, 2
    T = B * nodes
    mk = lambda *s: torch.tensor(r.standard_normal(s), dtype=torch.float32)      # noqa: E731
    q, k = (torch.nn.functional.normalize(mk(T, H, d), dim=-1).to(dtype) for _ in range(2))
    v, S = mk(T, H, d).to(dtype), mk(B, H, d, d)
    g = torch.tensor(np.stack([np.concatenate([gates(r, nodes, kind, strong) for _ in range(B)]) for _ in range(H)], 1))
    beta = torch.tensor(r.random((T, H)), dtype=torch.float32)
    # a chain, and a tree of branches from nodes above and below the gate
    parents = list(range(-1, nodes - 1)) + [-1] + [int(r.integers(max(0, i - 4), i)) for i in range(1, nodes)]
    cu = [0, nodes, T]
    out = gdn.gdn_tree_step(*(x.to(DEV) for x in (q, k, v, g, beta)), torch.tensor(parents, dtype=torch.int32, device=DEV),
                            S.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV))
    f64 = lambda x: x.detach().to("cpu", torch.float64).numpy()                  # noqa: E731
    ref = D.tree_step(*(f64(x) for x in (q, k, v, g, beta)), parents, f64(S), cu)
    bar = 2.0 ** -20 if dtype == torch.float32 else 2.0 ** -8 / 3 ** 0.5
    got = f64(out)
    for b in range(B):
        for h in range(H):
            at = slice(cu[b], cu[b + 1])
            err = np.linalg.norm(got[at, h] - ref[at, h]) / np.linalg.norm(ref[at, h])
            assert err <= bar, (b, h, err)
