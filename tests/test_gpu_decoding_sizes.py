"""Sizes that do not fit the C entry points' 32-bit integers are refused, not
cut to their low bits."""
import pytest
import torch

import linear_attention_vlm_b200 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 33 + 4, -2 ** 31 - 1, 10 ** 12])
def test_a_size_past_32_bits_is_refused(big):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(1, 8, 2, 128, dtype=torch.bfloat16, device="cuda")
    n, w, gates = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    state = torch.zeros(1, 2, 128, 128, device="cuda")
    with pytest.raises(ValueError, match="window"):
        gdn.gdn_tree_attention(x, x, x, None, c, c, n, window=big)
    with pytest.raises(ValueError, match="max_nodes"):
        gdn.gdn_tree_attention(x, x, x, None, c, c, n, max_nodes=big)
    with pytest.raises(ValueError, match="max_nodes"):
        gdn.gdn_tree_step(x, x, x, gates, gates, None, state, max_nodes=big)
    with pytest.raises(ValueError, match="window"):
        gdn.gdn_cache_weights(x, gates, x, c, w, n, window=big)
    with pytest.raises(ValueError, match="recent"):
        gdn.gdn_cache_insert(x, x, c, c.clone(), w, w.int(), n, n.clone(), recent=big)


def test_the_largest_window_is_none():
    # a window that reaches past every slot, up to the largest there is
    gen = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()      # noqa: E731
    q, k, v, kc, vc = bf(5, 4, 128), bf(5, 2, 128), bf(5, 2, 128), bf(1, 90, 2, 128), bf(1, 90, 2, 128)
    n, w = torch.tensor([90], dtype=torch.int32).cuda(), torch.zeros(1, 2, 90).cuda()
    o, lse = gdn.gdn_tree_attention(q, k, v, None, kc, vc, n)
    ref = gdn.gdn_cache_weights(q, lse, k, kc, w, n, weights_out=torch.empty_like(w))
    for window in (95, 2 ** 31 - 1):
        got = gdn.gdn_tree_attention(q, k, v, None, kc, vc, n, window=window)
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        got = gdn.gdn_cache_weights(q, lse, k, kc, w, n, window=window, weights_out=torch.empty_like(w))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
