"""The README's turn of drafted trees over a bounded cache, as it stands there."""
import ast
import os
import re

import pytest
import torch

import linear_attention_vlm_b200 as gdn

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def use_block():
    text = open(README).read()
    lines = re.search(r"## Use \(Python\)\n\n((?:    .*\n|\n)+)", text).group(1).splitlines()
    return "\n".join(x[4:] for x in lines)


def turn():
    """The calls over the cache, from the check of the drafts on."""
    block = use_block()
    return block[block.index("o, lse = gdn.gdn_tree_attention"):]


def keywords(name):
    calls = [n for n in ast.walk(ast.parse(turn())) if isinstance(n, ast.Call) and getattr(n.func, "attr", "") == name]
    assert len(calls) == 1
    return {k.arg: ast.unparse(k.value) for k in calls[0].keywords}


def test_weights_go_by_the_window_of_their_log_sum_exp():
    att, wts = keywords("gdn_tree_attention"), keywords("gdn_cache_weights")
    for name in ("cache_pos", "seen", "window", "scale"):
        assert att.get(name) == wts.get(name), name


def test_the_bound_of_the_nodes_is_given():
    # without it a batch of small trees runs with the bounds of 64 nodes
    assert "max_nodes" in keywords("gdn_tree_attention") and "max_nodes" in keywords("gdn_tree_step")


@pytest.mark.gpu
def test_the_turn_runs_and_its_weights_add_up():
    """All drafts accepted (chains): what the queries lay on slots and on one
    another is one for every query head, up to fp32 sums of bf16 scores (the exponents
    are off by 2^-23 128 |q| |k| / sqrt(128) < 2e-4)."""
    B, T, cap, n = 2, 6, 1100, 3
    gen = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()      # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()                   # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(s, generator=gen), dim=-1).to(torch.bfloat16).cuda()  # noqa: E731
    env = dict(gdn=gdn, q=bf(T, 16, 128), k=bf(T, 2, 128), v=bf(T, 2, 128), parents=ints([-1, 0, 1] * 2), cu=ints([0, 3, 6]),
               k_cache=bf(B, cap, 2, 128), v_cache=bf(B, cap, 2, 128), cache_lens=ints([cap, 300]), seen=ints([20000, 12000]),
               w=torch.zeros(B, 2, cap).cuda(), n=n,
               # kept slots, many of them from before the window
               pos=torch.randint(0, 12000, (B, 2, cap), generator=gen).to(torch.int32).cuda(),
               g=-torch.rand(T, 16, generator=gen).cuda(), beta=torch.rand(T, 16, generator=gen).cuda(),
               state=torch.randn(B, 16, 128, 128, generator=gen).cuda())
    env["qa"], env["ka"], env["va"], env["cu_a"] = (env[x] for x in ("q", "k", "v", "cu"))
    text = turn()
    last = text.index("w, pos, cache_lens, seen, slots")
    before = text[:last]
    check, rest = before.index("o = gdn.gdn_tree_step"), before.index("# then")
    exec(before[:check], env)
    lse = env["lse"]
    env.update(lse_a=lse)
    qkv = {x: env[x] for x in "qkv"}
    env.update(q=unit(T, 16, 128), k=unit(T, 16, 128), v=bf(T, 16, 128))
    exec(before[check:rest], env)
    env.update(qkv)
    exec(before[rest:], env)
    live = torch.arange(cap, device="cuda") < env["cache_lens"][:, None, None]
    total = (env["w"] * live).sum((1, 2)) + env["new_w"].sum(1).view(B, 3).sum(1)
    assert torch.allclose(total.cpu(), torch.full((B,), 3.0 * 16), rtol=2e-3)
    exec(text[last:], env)
    assert env["cache_lens"].tolist() == [cap, 303] and env["seen"].tolist() == [20003, 12003]
