"""Windows and positions beyond 2^30: the weights count the slots that the
attention counts."""
import numpy as np
import pytest
import torch

import linear_attention_vlm_b200 as gdn
from oracle import decoding as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [5, 1_000_000_000, 1_073_741_900, 1_700_000_000, 2_000_000_001, 2_147_483_646])
def test_far_positions(window):
    r = np.random.default_rng(0)
    gen = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16)             # noqa: E731
    n, Hq, Hkv, cap, seen = 3, 8, 2, 200, 2_000_000_000
    q, k, v, kc, vc = bf(n, Hq, 128), bf(n, Hkv, 128), bf(n, Hkv, 128), bf(1, cap, Hkv, 128), bf(1, cap, Hkv, 128)
    near = np.array([0, 1, seen - 1, seen - 4, seen - 5] + [max(0, seen - window + d) for d in range(-2, 5)])
    pos = np.concatenate([np.tile(near, (1, Hkv, 1)), r.integers(0, seen, (1, Hkv, cap - near.size))], -1)
    np64 = lambda x: x.detach().to("cpu", torch.float64).numpy()                 # noqa: E731
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()       # noqa: E731
    place = dict(cache_pos=ints(pos), seen=ints([seen]), window=window)
    _, lse = gdn.gdn_tree_attention(q.cuda(), k.cuda(), v.cuda(), None, kc.cuda(), vc.cuda(), ints([cap]), **place)
    _, ref_lse = D.tree_attention(np64(q), np64(k), np64(v), None, np64(kc), np64(vc), [cap], [0, n], pos, [seen], window)
    assert np.abs(np64(lse) - ref_lse).max() <= 1e-3       # scores are off by 2^-23 128 |q| |k| / sqrt(128)
    w, new = gdn.gdn_cache_weights(q.cuda(), lse, k.cuda(), kc.cuda(), torch.zeros(1, Hkv, cap).cuda(), ints([cap]), **place)
    ref, ref_new = D.cache_weights(np64(q), np64(lse), np64(k), np64(kc), np.zeros((1, Hkv, cap)), [cap], [0, n], [0, n], pos, [seen], window)
    assert np.allclose(np64(w), ref, rtol=2e-3, atol=0) and np.allclose(np64(new), ref_new, rtol=2e-3, atol=0)
