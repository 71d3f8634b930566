"""The bounded waits of the kernels over a cache: a wait that gives up leaves a
code in the workspace's first word and nothing in flight, and the next call
runs normally."""
import pytest
import torch

import linear_attention_vlm_b200 as gdn

pytestmark = pytest.mark.gpu


def inputs(nodes):
    gen = torch.Generator(device="cuda").manual_seed(0)
    bf = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    return (bf(nodes, 16, 128), bf(nodes, 2, 128), bf(nodes, 2, 128), None, bf(1, 4000, 2, 128), bf(1, 4000, 2, 128),
            torch.tensor([4000], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("nodes", [1, 64])
def test_attention_wait_that_gives_up(nodes):
    args = inputs(nodes)
    ws = torch.empty(gdn.gdn_tree_attention_workspace_size(1, nodes, nodes, 4000, 16, 2), dtype=torch.uint8, device="cuda")
    word = ws.view(torch.int32)
    ref = gdn.gdn_tree_attention(*args, workspace=ws)
    assert gdn.gdn_read_status(word) == 0
    try:
        gdn.gdn_set_wait_limit(0)
        gdn.gdn_tree_attention(*args, workspace=ws)
        assert gdn.gdn_read_status(word) != 0
    finally:
        gdn.gdn_set_wait_limit(gdn.WAIT_LIMIT_DEFAULT)
    got = gdn.gdn_tree_attention(*args, workspace=ws)
    assert gdn.gdn_read_status(word) == 0
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("nodes", [1, 64])
def test_weights_wait_that_gives_up(nodes):
    q, k, _, _, kc, _, lens = inputs(nodes)
    lse, w = torch.full((nodes, 16), 9.0, device="cuda"), torch.zeros(1, 2, 4000, device="cuda")
    ws = torch.empty(gdn.gdn_cache_weights_workspace_size(1, nodes, nodes, 4000, 16, 2), dtype=torch.uint8, device="cuda")
    word = ws.view(torch.int32)
    run = lambda: gdn.gdn_cache_weights(q, lse, k, kc, w, lens, weights_out=torch.empty_like(w), workspace=ws)  # noqa: E731
    ref = run()
    assert gdn.gdn_read_status(word) == 0
    try:
        gdn.gdn_set_wait_limit(0)
        run()
        assert gdn.gdn_read_status(word) != 0
    finally:
        gdn.gdn_set_wait_limit(gdn.WAIT_LIMIT_DEFAULT)
    got = run()
    assert gdn.gdn_read_status(word) == 0
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
