"""fp64 CPU oracle of decoding over trees of drafted tokens and a cache of
constant size -- TEST INFRASTRUCTURE ONLY (same rules as the rest of
``oracle``).

Plain numpy float64, one sequence, head and node at a time, written from the
definitions in include/gdn.h.  A node's parent is an index inside its
sequence that is smaller than its own; any other value means that the node
continues the tokens already seen.
"""
from __future__ import annotations

import math
from typing import List, Optional

import numpy as np


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def paths(parents, n: int) -> List[List[int]]:
    """Every node's line of ancestors, itself last; ``parents`` None: a chain."""
    lines: List[List[int]] = []
    for i in range(n):
        p = i - 1 if parents is None else int(parents[i])
        lines.append((lines[p] if 0 <= p < i else []) + [i])
    return lines


def tree_attention(q, k, v, parents, k_cache, v_cache, lens, cu, pos=None, seen=None, window: int = 0,
                   scale: Optional[float] = None):
    """q [T, Hq, d]; k, v [T, Hkv, d]; caches [B, cap, Hkv, d]; lens [B]; pos
    [B, Hkv, cap].  Returns (o, lse)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    Hq, d = q.shape[1:]
    grp = Hq // k.shape[1]
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    for b in range(len(cu) - 1):
        t0, n, l = int(cu[b]), int(cu[b + 1] - cu[b]), int(lens[b])
        lines = paths(None if parents is None else parents[t0:t0 + n], n)
        before = l if pos is None else int(seen[b])
        for h in range(Hq):
            kh = h // grp
            old_k, old_v = _f64(k_cache[b][:l, kh]), _f64(v_cache[b][:l, kh])
            place = np.arange(l) if pos is None else np.asarray(pos[b][kh][:l], dtype=np.int64)
            for i, line in enumerate(lines):
                here = before + len(line) - 1
                near = np.ones(l, bool) if not window else here - place < window
                own = [t0 + j for j in (line if not window else line[-window:])]
                keys = np.concatenate([old_k[near], k[own, kh]])
                vals = np.concatenate([old_v[near], v[own, kh]])
                x = keys @ q[t0 + i, h] * sc
                e = np.exp(x - x.max())
                o[t0 + i, h] = (e / e.sum()) @ vals
                lse[t0 + i, h] = x.max() + math.log(e.sum())
    return o, lse


def tree_step(q, k, v, g, beta, parents, state, cu):
    """q, k, v [T, H, d]; g, beta [T, H]; state [B, H, dv, dk].  Returns out."""
    q, k, v, g, beta, state = (_f64(x) for x in (q, k, v, g, beta, state))
    out = np.zeros_like(v)
    for b in range(len(cu) - 1):
        t0, n = int(cu[b]), int(cu[b + 1] - cu[b])
        for h in range(q.shape[1]):
            states: List[np.ndarray] = []
            for i in range(n):
                t = t0 + i
                p = i - 1 if parents is None else int(parents[t])
                S = np.exp(g[t, h]) * (states[p] if 0 <= p < i else state[b, h])
                S = S + np.outer(beta[t, h] * (v[t, h] - S @ k[t, h]), k[t, h])
                out[t, h] = S @ q[t, h]
                states.append(S)
    return out


def cache_weights(q, lse, k, k_cache, weights, lens, cu_q, cu, pos=None, seen=None, window: int = 0,
                  scale: Optional[float] = None):
    """q [Tq, Hq, d]; lse [Tq, Hq]; k [T, Hkv, d]; weights [B, Hkv, cap].
    Returns (weights, new_weights [T, Hkv])."""
    q, lse, k = _f64(q), _f64(lse), _f64(k)
    w, new = _f64(weights).copy(), np.zeros(k.shape[:2])
    grp, d = q.shape[1] // k.shape[1], q.shape[2]
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    for b in range(len(cu) - 1):
        t0, m, l = int(cu[b]), int(cu[b + 1] - cu[b]), int(lens[b])
        nq = min(int(cu_q[b + 1] - cu_q[b]), m)
        q0 = int(cu_q[b + 1]) - nq
        before = l if pos is None else int(seen[b])
        for kh in range(k.shape[1]):
            old_k = _f64(k_cache[b][:l, kh])
            place = np.arange(l) if pos is None else np.asarray(pos[b][kh][:l], dtype=np.int64)
            for i in range(nq):
                mine = m - nq + i
                lo = 0 if not window else max(0, mine - window + 1)
                near = np.ones(l, bool) if not window else before + mine - place < window
                for h in range(kh * grp, (kh + 1) * grp):
                    if lse[q0 + i, h] == -np.inf:
                        continue
                    w[b, kh, :l][near] += np.exp(old_k[near] @ q[q0 + i, h] * sc - lse[q0 + i, h])
                    new[t0 + lo:t0 + mine + 1, kh] += np.exp(k[t0 + lo:t0 + mine + 1, kh] @ q[q0 + i, h] * sc - lse[q0 + i, h])
    return w, new


def cache_insert(weights, pos, lens, seen, cu, recent: int, capacity: int, new_weights=None):
    """Which tokens go where.  Returns (weights, pos, lens, seen, slots
    [T, Hkv]); keys and values follow ``slots``."""
    w, pos = np.array(weights, dtype=np.float32), np.array(pos, dtype=np.int64)
    T, Hkv = int(cu[-1]), w.shape[1]
    new_weights = None if new_weights is None else np.asarray(new_weights)
    lens_out, seen_out = np.array(lens, dtype=np.int64), np.array(seen, dtype=np.int64)
    slots = np.full((T, Hkv), -1, dtype=np.int64)
    for b in range(len(cu) - 1):
        t0, m, l = int(cu[b]), int(cu[b + 1] - cu[b]), int(lens[b])
        room, end = min(capacity, l + m), int(seen[b]) + m
        lens_out[b], seen_out[b] = room, end
        for h in range(Hkv):
            cand = [(float(w[b, h, s]), int(pos[b, h, s])) for s in range(l)]
            cand += [(0.0 if new_weights is None else float(new_weights[t0 + j, h]), int(seen[b]) + j) for j in range(m)]

            def rank(i):   # recent first, then heavy, then early; NaN last
                weight, place = cand[i]
                young = end - place <= recent
                bad = weight != weight
                return (not young, 0.0 if young else (math.inf if bad else -weight), 0 if young else bad, i)

            kept = set(sorted(range(l + m), key=rank)[:room])
            free = [s for s in range(room) if s >= l or s not in kept]
            for i, s in zip([i for i in range(l, l + m) if i in kept], free):
                w[b, h, s], pos[b, h, s] = cand[i]
                slots[t0 + i - l, h] = s
    return w, pos, lens_out, seen_out, slots
