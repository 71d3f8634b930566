"""The oracle of decoding over drafted trees and a bounded cache, pinned by
what its definitions imply: a chain is the sequential recurrence and the
causal window attention, a node's result is that of its own path, attention
weights of a query add up to one, a cache that only keeps the recent is a
sliding window."""
import numpy as np
import pytest

import oracle
from oracle import decoding as D


def rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def tree(seed, n):
    r = np.random.default_rng(seed)
    return np.array([r.integers(-1, i) if i else -1 for i in range(n)])


def unit(x):
    return x / np.linalg.norm(x, axis=-1, keepdims=True)


def gdn_inputs(seed, T, H, d):
    return (unit(rand(seed, T, H, d)), unit(rand(seed + 1, T, H, d)), rand(seed + 2, T, H, d),
            -0.1 * np.abs(rand(seed + 3, T, H)), 1 / (1 + np.exp(-rand(seed + 4, T, H))))


def test_chain_step_is_the_recurrence():
    q, k, v, g, b = gdn_inputs(0, 9, 2, 8)
    S = rand(9, 2, 2, 8, 8)
    cu = [0, 4, 9]
    out = D.tree_step(q, k, v, g, b, None, S, cu)
    ref, _ = oracle.prefill(q, k, v, g, b, S, cu)
    assert np.allclose(out, ref, rtol=0, atol=1e-12)


def test_step_of_a_node_is_that_of_its_path():
    n = 12
    q, k, v, g, b = gdn_inputs(5, n, 1, 8)
    S, parents = rand(4, 1, 1, 8, 8), tree(3, n)
    out = D.tree_step(q, k, v, g, b, parents, S, [0, n])
    for i, line in enumerate(D.paths(parents, n)):
        ref, _ = oracle.prefill(q[line], k[line], v[line], g[line], b[line], S, [0, len(line)])
        assert np.allclose(out[i], ref[-1], rtol=0, atol=1e-12)


def test_the_closed_form_over_ancestors():
    # (I + A) U = beta (V - exp(G) K S^T), o = exp(G) Q S^T + (decay q.k) U over ancestors
    n, d = 17, 8
    q, k, v, g, b = (x[:, 0] for x in gdn_inputs(20, n, 1, d))
    S, parents = rand(8, d, d), tree(6, n)
    anc = np.zeros((n, n), bool)
    for i, line in enumerate(D.paths(parents, n)):
        anc[i, line] = True
    G = anc @ g
    decay = np.where(anc, np.exp(np.where(anc, G[:, None] - G[None], 0)), 0)
    A = b[:, None] * decay * (k @ k.T) * (1 - np.eye(n))
    U = np.linalg.solve(np.eye(n) + A, b[:, None] * (v - np.exp(G)[:, None] * (k @ S.T)))
    o = np.exp(G)[:, None] * (q @ S.T) + (decay * (q @ k.T)) @ U
    ref = D.tree_step(q[:, None], k[:, None], v[:, None], g[:, None], b[:, None], parents, S[None, None], [0, n])
    assert np.allclose(o, ref[:, 0], rtol=0, atol=1e-11)


@pytest.mark.parametrize("window", [1, 3, 6, 100])
def test_chain_attention_is_causal_window_attention(window):
    T, cut = 14, 9
    q, k, v = rand(1, T, 4, 8), rand(2, T, 2, 8), rand(3, T, 2, 8)
    ref = oracle.swa_attention(q, k, v, window=window)
    o, _ = D.tree_attention(q[cut:], k[cut:], v[cut:], None, k[None, :cut], v[None, :cut], [cut], [0, T - cut],
                            window=window)
    assert np.allclose(o, ref[cut:], rtol=0, atol=1e-13)


def test_attention_does_not_depend_on_the_order_of_slots():
    n, l = 6, 11
    q, k, v = rand(1, n, 2, 8), rand(2, n, 1, 8), rand(3, n, 1, 8)
    kc, vc = rand(4, 1, l, 1, 8), rand(5, 1, l, 1, 8)
    parents, order = tree(1, n), np.random.default_rng(2).permutation(l)
    a = D.tree_attention(q, k, v, parents, kc, vc, [l], [0, n], window=5)
    b = D.tree_attention(q, k, v, parents, kc[:, order], vc[:, order], [l], [0, n], pos=order[None, None], seen=[l],
                         window=5)
    assert np.allclose(a[0], b[0], atol=1e-13) and np.allclose(a[1], b[1], atol=1e-13)


def test_weights_of_a_query_add_up_to_one():
    n, l, Hq, Hkv = 5, 7, 4, 2
    q, k, v = rand(1, n, Hq, 8), rand(2, n, Hkv, 8), rand(3, n, Hkv, 8)
    kc = rand(4, 1, l, Hkv, 8)
    _, lse = D.tree_attention(q, k, v, None, kc, kc, [l], [0, n])
    w, new = D.cache_weights(q, lse, k, kc, np.zeros((1, Hkv, l)), [l], [0, n], [0, n])
    assert np.allclose(w.sum(-1)[0] + new.sum(0), n * Hq / Hkv)
    # the last query alone
    w, new = D.cache_weights(q[-1:], lse[-1:], k, kc, np.ones((1, Hkv, l)), [l], [0, 1], [0, n])
    assert np.allclose((w - 1).sum(-1)[0] + new.sum(0), Hq / Hkv)


def test_keeping_the_recent_is_a_sliding_window():
    cap, H = 5, 2
    w, pos = np.zeros((1, H, cap)), np.zeros((1, H, cap))
    lens, seen = [0], [0]
    r = np.random.default_rng(0)
    for m in (3, 1, 4, 0, 9, 2):
        w, pos, lens, seen, slots = D.cache_insert(w, pos, lens, seen, [0, m], cap, cap, r.random((m, H)))
        for h in range(H):
            assert sorted(pos[0, h, :lens[0]]) == list(range(max(0, seen[0] - cap), seen[0]))


def test_eviction_by_weight_by_hand():
    # slots of weight 5, 1, 3, 1 at positions 0..3; tokens 4, 5 of weight 0 and 4
    w, pos, lens, seen, slots = D.cache_insert([[[5., 1., 3., 1.]]], [[[0, 1, 2, 3]]], [4], [4], [0, 2], 0, 4, [[0.], [4.]])
    # the four heaviest: 5, 4, 3 and the earlier of the two ones
    assert slots.tolist() == [[-1], [3]] and pos[0, 0].tolist() == [0, 1, 2, 5] and lens.tolist() == [4] and seen.tolist() == [6]
    # with the last three positions protected (3, 4, 5) only one place is left, for the heaviest
    w, pos, lens, seen, slots = D.cache_insert([[[5., 1., 3., 1.]]], [[[0, 1, 2, 3]]], [4], [4], [0, 2], 3, 4, [[0.], [4.]])
    assert slots.tolist() == [[1], [2]] and pos[0, 0].tolist() == [0, 4, 5, 3]
    assert w[0, 0].tolist() == [5., 0., 4., 1.]
