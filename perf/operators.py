"""Timed cases of the decoding operators over drafted trees and bounded caches.

Four operators of a hybrid block (Gated DeltaNet layers between attention layers) that verifies trees of
drafted tokens and keeps a cache of constant size:

  attention   tree nodes attend to a cache and to their ancestors          (gdn_tree_attention)
  step        the Gated DeltaNet read-out of every tree node from a state  (gdn_tree_step)
  weights     attention weights of tokens added up per cache slot          (gdn_cache_weights)
  insert      tokens enter a full cache in place of the lightest slots     (gdn_cache_insert)

``run`` computes an operator in elementary torch operations, or, with ``own`` set, through the package.
"""
import math
import random

import torch

own = False

D = 128                 # head dimension of the attention cases
ROW = D * 2             # bytes of one cached key or value (bf16)
HEADS = ((16, 2), (16, 16), (12, 4), (8, 1), (32, 8), (5, 5), (24, 2))


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of one sequence against a full window: the latency of plain decoding
        dict(name="attention token", op="attention", seqs=1, nodes=1, cache=8192, hq=16, hkv=2, window=0),
        # one token for each of a serving batch with caches of all lengths
        dict(name="attention batch", op="attention", seqs=64, nodes=1, cache=8192, hq=16, hkv=2, window=0),
        # large draft trees over ring caches that hold exactly the window, masked by position
        dict(name="attention trees", op="attention", seqs=32, nodes=64, cache=8192, hq=16, hkv=2, window=8192),
        # a middling tree at the end of a very long context
        dict(name="attention long", op="attention", seqs=1, nodes=24, cache=262144, hq=16, hkv=2, window=0),
        # a small tree of one sequence through a Gated DeltaNet layer
        dict(name="step tree", op="step", seqs=1, nodes=7, heads=16, d=128, f32=False),
        # a serving batch of trees
        dict(name="step batch", op="step", seqs=64, nodes=16, heads=16, d=128, f32=False),
        # fp32 and d = 64, as the tiny workload has them
        dict(name="step fp32", op="step", seqs=24, nodes=33, heads=12, d=64, f32=True),
        # the accepted tokens of a batch, weighed over their caches
        dict(name="weights accepted", op="weights", seqs=32, queries=5, tokens=5, cache=8192, hq=16, hkv=2, window=0),
        # the last tokens of a long prompt weigh the prompt before it is cut down to the cache
        dict(name="weights prompt", op="weights", seqs=1, queries=64, tokens=32768, cache=8, hq=16, hkv=2, window=0),
        # accepted tokens of a batch enter full caches
        dict(name="insert accepted", op="insert", seqs=64, tokens=4, cache=8192, hkv=2, recent=1024),
        # one video frame a stream (274 tokens)
        dict(name="insert frame", op="insert", seqs=16, tokens=274, cache=8192, hkv=2, recent=2048),
        # a prompt cut down to the cache in one go
        dict(name="insert prompt", op="insert", seqs=1, tokens=32768, cache=8192, hkv=2, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(("attention", "step", "weights", "insert"))
    hq, hkv = rng.choice(HEADS)
    if op == "attention":
        cache = _log(rng, 1, 262144)
        return dict(op=op, seqs=_log(rng, 1, 128), nodes=_log(rng, 1, 64), cache=cache, hq=hq, hkv=hkv,
                    window=rng.choice((0, 0, cache, max(1, cache // 3))))
    if op == "step":
        return dict(op=op, seqs=_log(rng, 1, 128), nodes=_log(rng, 1, 64), heads=rng.choice((1, 3, 12, 16)),
                    d=rng.choice((64, 128)), f32=rng.random() < 0.3)
    if op == "weights":
        if rng.random() < 0.5:
            m = _log(rng, 1, 64)
            cache = _log(rng, 1, 65536)
            return dict(op=op, seqs=_log(rng, 1, 64), queries=m, tokens=m, cache=cache, hq=hq, hkv=hkv,
                        window=rng.choice((0, cache)))
        tokens = _log(rng, 64, 32768)
        return dict(op=op, seqs=rng.randint(1, 4), queries=rng.randint(1, 64), tokens=tokens, cache=8, hq=hq, hkv=hkv,
                    window=0)
    cache = _log(rng, 1, 32768)
    return dict(op=op, seqs=_log(rng, 1, 64), tokens=_log(rng, 1, 16384), cache=cache, hkv=hkv,
                recent=rng.randint(0, cache))


def _memory(case):
    """Bytes of the largest tensors that a plain pass makes."""
    if case["op"] == "insert":
        return 96 * case["seqs"] * case["hkv"] * (case["cache"] + case["tokens"]) + 4 * ROW * case["seqs"] * case["hkv"] * (case["cache"] + case["tokens"])
    if case["op"] == "step":
        return 12 * case["seqs"] * case["heads"] * case["d"] ** 2
    rows = case["seqs"] * case["hq"] * (case["nodes"] if case["op"] == "attention" else case["queries"])
    keys = case["cache"] + (case["nodes"] if case["op"] == "attention" else case["tokens"])
    return 16 * rows * keys + 3 * ROW * case["seqs"] * case["hkv"] * keys


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        case = _draw(rng)
        w = work(case)
        b, f = most[case["op"]]
        if w["bytes"] <= b and w["flops"] <= f and _memory(case) <= 12e9:
            return case


# ---------------------------------------------------------------- sizes of one case

def _sizes(case):
    """Lengths of a case's sequences, from its sizes alone: {"new": tokens or nodes, "queries", "lens": cached}."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    B, n = case["seqs"], case.get("nodes", case.get("tokens"))
    ragged = lambda lo, hi: [hi if b == 0 else rng.randint(lo, hi) for b in range(B)]  # noqa: E731
    new = ragged(max(1, n // 2), n)
    out = dict(new=new)
    if case["op"] == "step":
        return out
    L = case["cache"]
    if case["op"] == "insert":
        out["lens"] = [L] * B if n < L else [0] * B        # a full cache, or a prompt into an empty one
    elif case["op"] == "weights":
        out["lens"] = ragged((L + 1) // 2, L) if L > 8 else [0] * B
        out["queries"] = [min(case["queries"], m) for m in new]
    else:
        out["lens"] = [L] * B if case["window"] else ragged(min(L, 16), L)
    return out


def work(case):
    z = _sizes(case)
    T, B = sum(z["new"]), case["seqs"]
    if case["op"] == "step":
        H, d, es = case["heads"], case["d"], 4 if case["f32"] else 2
        nodes = 4 * d * d + 3 * d                                  # two reads of the state and the write
        pairs = sum(n * (n + 1) // 2 for n in z["new"]) * 8 * d     # products with the nodes before
        return dict(bytes=B * H * d * d * 4 + 4 * T * H * d * es + 8 * T * H + 4 * T, flops=H * (T * nodes + pairs))
    if case["op"] == "insert":
        H, L = case["hkv"], case["cache"]
        moved = sum(min(m, L) for m in z["new"])
        slots = sum(min(L, l + m) for l, m in zip(z["lens"], z["new"]))
        return dict(bytes=4 * moved * H * ROW + H * 8 * (sum(z["lens"]) + slots) + 8 * T * H, flops=H * (sum(z["lens"]) + T))
    Hq, Hkv = case["hq"], case["hkv"]
    slots = sum(z["lens"])
    pos = 4 * slots * Hkv if case["window"] else 0
    if case["op"] == "attention":
        pairs = sum(n * (l + (n + 1) // 2) for n, l in zip(z["new"], z["lens"]))
        return dict(bytes=2 * T * (Hq + Hkv) * ROW + 2 * slots * Hkv * ROW + 4 * T * Hq + pos, flops=4 * D * Hq * pairs)
    pairs = sum(q * (l + m - q // 2) for q, m, l in zip(z["queries"], z["new"], z["lens"]))
    Q = sum(z["queries"])
    return dict(bytes=Q * Hq * (ROW + 4) + (T + slots) * Hkv * ROW + 8 * slots * Hkv + 4 * T * Hkv + pos, flops=2 * D * Hq * pairs)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda"
    z = _sizes(case)
    B, T = case["seqs"], sum(z["new"])
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = random.Random(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)                   # noqa: E731
    bf16 = lambda *shape: torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)                          # noqa: E731
    cu = lambda v: ints([sum(v[:i]) for i in range(B + 1)])                                  # noqa: E731
    s = dict(op=case["op"], cu=cu(z["new"]))
    if case["op"] in ("attention", "step"):
        s["nodes"] = case["nodes"]
        s["parents"] = ints([rng.randint(max(-1, i - 6), i - 1) if i else -1 for n in z["new"] for i in range(n)])
    if case["op"] == "step":
        H, d, dt = case["heads"], case["d"], torch.float32 if case["f32"] else torch.bfloat16
        unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)                           # noqa: E731
        s.update(q=unit(normal(T, H, d)), k=unit(normal(T, H, d)), v=normal(T, H, d).to(dt),
                 g=-0.05 * torch.nn.functional.softplus(normal(T, H)), beta=torch.sigmoid(normal(T, H)),
                 state=0.1 * normal(B, H, d, d))
        return s
    L, Hkv = case["cache"], case["hkv"]
    s.update(k=bf16(T, Hkv, D), v=bf16(T, Hkv, D), k_cache=bf16(B, L, Hkv, D), lens=ints(z["lens"]))
    if case["op"] != "weights":
        s["v_cache"] = bf16(B, L, Hkv, D)
    # tokens of the stream so far; a slot's position: the last `cache` ones, in a ring
    seen = [l + (rng.randint(0, 100000) if l == L else 0) for l in z["lens"]]
    s["seen"] = ints(seen)
    slot = torch.arange(L, device=dev)
    last = s["seen"].long()[:, None] - 1
    pos = torch.where(s["lens"][:, None] == L, last - (last - slot) % L, slot).to(torch.int32)
    s["pos"] = pos[:, None].expand(B, Hkv, L).contiguous()
    if case["op"] == "insert":
        # heavy-tailed sums, many slots that nothing has looked at yet
        w = torch.relu(normal(B, Hkv, L)) ** 4
        s.update(weights=w, new_weights=torch.relu(normal(T, Hkv)) ** 4, recent=case["recent"], tokens=case["tokens"])
        s["outs"] = [w.clone(), s["pos"].clone(), torch.empty_like(s["lens"]), torch.empty_like(s["seen"])]
        return s
    s["window"] = case["window"]
    if case["op"] == "attention":
        s["q"] = bf16(T, case["hq"], D)
        return s
    s["cu_q"], s["queries"], s["tokens"] = cu(z["queries"]), case["queries"], case["tokens"]
    s["q"] = bf16(sum(z["queries"]), case["hq"], D)
    # log-sum-exp of scores of q with normal keys, as the attention pass leaves it
    keys = torch.tensor([l + m for l, m in zip(z["lens"], z["new"])], device=dev, dtype=torch.float32)
    keys = keys.repeat_interleave(torch.tensor(z["queries"], device=dev))
    s["lse"] = keys.log()[:, None] + s["q"].float().square().sum(-1) / (2 * D)
    s["weights"] = torch.relu(normal(B, Hkv, L)) ** 4
    s["out"] = s["weights"].clone()
    return s


# ---------------------------------------------------------------- plain forms (fp32)

def _padded(cu, n, T):
    """Rows [B, n] of a packed tensor, and which of them exist."""
    at = cu[:-1, None].long() + torch.arange(n, device=cu.device)
    there = at < cu[1:, None]
    return at.clamp(max=max(T - 1, 0)), there


def _ancestors(parents, at, there):
    """[B, n, n] whether node j is node i or one of its ancestors, and depths [B, n]."""
    n = at.shape[1]
    up = torch.where(there, parents[at].long(), -1)
    step = torch.eye(n, device=at.device, dtype=torch.float64) + (up[..., None] == torch.arange(n, device=at.device))
    anc = torch.linalg.matrix_power(step, max(n - 1, 1)) > 0
    return anc, anc.sum(-1) - 1


def _attention(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"]
    (T, Hq, _), Hkv, B, L, n = q.shape, k.shape[1], s["k_cache"].shape[0], s["k_cache"].shape[1], s["nodes"]
    at, there = _padded(cu, n, T)
    anc, depth = _ancestors(s["parents"], at, there)
    qp = q[at].float().view(B, n, Hkv, Hq // Hkv, D)
    old = torch.einsum("bnkgd,bskd->bkgns", qp, s["k_cache"].float()) / math.sqrt(D)
    new = torch.einsum("bnkgd,bmkd->bkgnm", qp, k[at].float()) / math.sqrt(D)
    sees = (torch.arange(L, device=q.device) < s["lens"][:, None])[:, None, None, None]     # [B, 1, 1, 1, L]
    if s["window"]:
        anc = anc & (depth[:, :, None] - depth[:, None, :] < s["window"])
        far = (s["seen"].long()[:, None] + depth)[:, None, :, None] - s["pos"].long()[:, :, None, :]
        sees = sees & (far < s["window"])[:, :, None]
    x = torch.cat([old.masked_fill_(~sees, -math.inf), new.masked_fill_(~anc[:, None, None], -math.inf)], -1)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    values = torch.cat([s["v_cache"].float(), v[at].float()], 1)
    o = torch.einsum("bkgns,bskd->bnkgd", x / total, values)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    return o[there].reshape(T, Hq, D).to(q.dtype), lse[there].reshape(T, Hq)


def _step(s):
    q, k, v, g, beta = (s[x] for x in ("q", "k", "v", "g", "beta"))
    T, n = q.shape[0], s["nodes"]
    at, there = _padded(s["cu"], n, T)
    anc, _ = _ancestors(s["parents"], at, there)
    heads = lambda x: x[at].float().transpose(1, 2)                                         # noqa: E731  [B, H, n, ...]
    q_, k_, v_ = heads(q), heads(k), heads(v)
    b_ = heads(beta)[..., None]
    G = torch.einsum("bij,bhj->bhi", anc.double(), heads(g).double())
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~anc[:, None], -math.inf).exp().float()
    gamma = G.exp().float()[..., None]
    reads = (q_ @ k_.transpose(-1, -2)) * decay
    eye = torch.eye(n, device=q.device)
    erase = (b_ * (k_ @ k_.transpose(-1, -2)) * decay * (1 - eye)).double()
    # (1 + A)^-1 = (1 - A)(1 + A^2)(1 + A^4) ..., A^64 = 0
    a2 = erase @ erase
    a4 = a2 @ a2
    a8 = a4 @ a4
    a16 = a8 @ a8
    a32 = a16 @ a16
    u = b_ * (v_ - gamma * (k_ @ s["state"].transpose(-1, -2)))
    u = u.double()
    u = u + a32 @ u
    u = u + a16 @ u
    u = u + a8 @ u
    u = u + a4 @ u
    u = u + a2 @ u
    u = (u - erase @ u).float()
    o = gamma * (q_ @ s["state"].transpose(-1, -2)) + reads @ u
    return o.transpose(1, 2)[there].to(q.dtype)


def _weights(s):
    q, k, B, L = s["q"], s["k"], s["k_cache"].shape[0], s["k_cache"].shape[1]
    (Q, Hq, _), (T, Hkv, _) = q.shape, k.shape
    aq, is_q = _padded(s["cu_q"], s["queries"], Q)
    ak, is_k = _padded(s["cu"], s["tokens"], T)
    m, nq = (s["cu"][1:] - s["cu"][:-1]).long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    rank = (m - nq)[:, None] + torch.arange(s["queries"], device=q.device)                   # a query's place among the tokens
    qp = q[aq].float().view(B, -1, Hkv, Hq // Hkv, D)
    lse = s["lse"][aq].view(B, -1, Hkv, Hq // Hkv).permute(0, 2, 3, 1)[..., None]
    old = torch.einsum("bnkgd,bskd->bkgns", qp, s["k_cache"].float()) / math.sqrt(D)
    new = torch.einsum("bnkgd,bmkd->bkgnm", qp, k[ak].float()) / math.sqrt(D)
    at = torch.arange(s["tokens"], device=q.device)
    reach = rank[:, :, None] - at
    sees_new = (reach >= 0) & is_q[..., None] & is_k[:, None, :]
    sees_old = (is_q[..., None] & (torch.arange(L, device=q.device) < s["lens"][:, None])[:, None, :])[:, None]
    if s["window"]:
        sees_new = sees_new & (reach < s["window"])
        far = (s["seen"].long()[:, None] + rank)[:, None, :, None] - s["pos"].long()[:, :, None, :]
        sees_old = sees_old & (far < s["window"])
    old = old.sub_(lse).exp_().masked_fill_(~sees_old[:, :, None], 0).sum((2, 3))
    new = new.sub_(lse).exp_().masked_fill_(~sees_new[:, None, None], 0).sum((2, 3))
    return s["weights"] + old, new.transpose(1, 2)[is_k]


def _insert(s):
    k, v, w, pos, lens, seen = (s[x] for x in ("k", "v", "weights", "pos", "lens", "seen"))
    (T, H, _), (B, _, L) = k.shape, w.shape
    m = (s["cu"][1:] - s["cu"][:-1]).long()
    M = s["tokens"]
    at, there = _padded(s["cu"], M, T)
    arange = torch.arange(L, device=k.device)
    cached = arange < lens[:, None]                                                          # [B, L]
    total = (seen + m)[:, None, None]
    age = torch.cat([total - pos, (m[:, None] - torch.arange(M, device=k.device))[:, None].expand(B, H, M)], -1)
    heavy = torch.cat([w, s["new_weights"][at].transpose(1, 2)], -1)
    exists = torch.cat([cached, there], -1)[:, None]
    # weights are >= 0, where the order of the bits is the order of the values; recent tokens stand above all
    key = torch.where(age <= s["recent"], 1 << 31, heavy.contiguous().view(torch.int32).long()).masked_fill(~exists, -1)
    order = key.argsort(dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, torch.arange(L + M, device=k.device).expand_as(order))
    keep = (lens + m).clamp(max=L)[:, None, None]
    stays = (rank < keep) & exists
    free = ~stays[..., :L] & (arange < keep)                                                 # evicted and empty slots
    enters = stays[..., L:]
    slot_of = (~free).long().argsort(dim=-1, stable=True)    # free slots first, ascending
    nth = (enters.long().cumsum(-1) - 1).clamp(min=0, max=L - 1)
    slots = torch.where(enters, slot_of.gather(-1, nth), -1)                                 # [B, H, M]
    b, h, j = enters.nonzero(as_tuple=True)
    to, row = slots[b, h, j], at[b, j]
    s["k_cache"][b, to, h] = k[row, h]
    s["v_cache"][b, to, h] = v[row, h]
    new_w, new_pos = w.clone(), pos.clone()
    new_w[b, h, to] = s["new_weights"][row, h]
    new_pos[b, h, to] = (seen[b] + j).to(torch.int32)
    return (s["k_cache"], s["v_cache"], new_w, new_pos, keep.view(B).to(torch.int32), (seen + m).to(torch.int32),
            slots.transpose(1, 2)[there].to(torch.int32))


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        return {"attention": _attention, "step": _step, "weights": _weights, "insert": _insert}[s["op"]](s)
    import linear_attention_vlm_b200 as gdn
    if s["op"] == "attention":
        ring = dict(cache_pos=s["pos"], seen=s["seen"], window=s["window"]) if s["window"] else {}
        return gdn.gdn_tree_attention(s["q"], s["k"], s["v"], s["parents"], s["k_cache"], s["v_cache"], s["lens"], s["cu"],
                                      max_nodes=s["nodes"], **ring)
    if s["op"] == "step":
        return gdn.gdn_tree_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parents"], s["state"], s["cu"],
                                 max_nodes=s["nodes"])
    if s["op"] == "weights":
        ring = dict(cache_pos=s["pos"], seen=s["seen"], window=s["window"]) if s["window"] else {}
        return gdn.gdn_cache_weights(s["q"], s["lse"], s["k"], s["k_cache"], s["weights"], s["lens"], s["cu_q"], s["cu"],
                                     weights_out=s["out"], **ring)
    w, pos, lens, seen = s["outs"]
    got = gdn.gdn_cache_insert(s["k"], s["v"], s["k_cache"], s["v_cache"], s["weights"], s["pos"], s["lens"], s["seen"],
                               s["cu"], recent=s["recent"], new_weights=s["new_weights"], weights_out=w, pos_out=pos,
                               lens_out=lens, seen_out=seen)
    return (s["k_cache"], s["v_cache"]) + tuple(got)


# ---------------------------------------------------------------- the definition in 64 bits, one sequence at a time

def exact(case, seed):
    s = prepare(case, seed)
    z = _sizes(case)
    starts = [sum(z["new"][:b]) for b in range(case["seqs"])]
    parents = s["parents"].tolist() if "parents" in s else None
    if case["op"] == "step":
        q, k, v = (s[x].double() for x in ("q", "k", "v"))
        alpha, beta = s["g"].double().exp(), s["beta"].double()
        out = torch.empty_like(v)
        for b, (t0, n) in enumerate(zip(starts, z["new"])):
            states = []
            for i in range(n):
                t, p = t0 + i, parents[t0 + i]
                S = (s["state"][b].double() if p < 0 else states[p]) * alpha[t][:, None, None]
                err = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
                S = S + err[:, :, None] * k[t][:, None, :]
                out[t] = torch.einsum("hvk,hk->hv", S, q[t])
                states.append(S)
        return out
    if case["op"] == "insert":
        return _exact_insert(s, z, starts)
    Hq, Hkv, scale, window = case["hq"], case["hkv"], D ** -0.5, case["window"] or 1 << 40
    shared = torch.arange(Hq, device="cuda") // (Hq // Hkv)      # the key head of a query head
    if case["op"] == "attention":
        out, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        for b, (t0, n, l) in enumerate(zip(starts, z["new"], z["lens"])):
            lines = []
            for i in range(n):
                lines.append((lines[parents[t0 + i]] if parents[t0 + i] >= 0 else []) + [i])
            here = torch.zeros(n, n, dtype=torch.bool)
            for i, line in enumerate(lines):
                here[i, line[-min(window, len(line)):]] = True
            place = s["seen"][b].item() + torch.tensor([len(x) - 1 for x in lines], device="cuda")
            for h in range(Hkv):
                mine = (shared == h).nonzero().view(-1)
                keys = torch.cat([s["k_cache"][b, :l, h], s["k"][t0:t0 + n, h]]).double()
                vals = torch.cat([s["v_cache"][b, :l, h], s["v"][t0:t0 + n, h]]).double()
                near = place[:, None] - s["pos"][b, h, :l].long() < window
                sees = torch.cat([near, here.cuda()], 1)[:, None, :]
                x = (s["q"][t0:t0 + n][:, mine].double() @ keys.T * scale).masked_fill(~sees, -math.inf)
                total = torch.logsumexp(x, -1)
                out[t0:t0 + n, mine] = torch.exp(x - total[..., None]) @ vals
                lse[t0:t0 + n, mine] = total
        return out, lse
    old, new = s["weights"].double(), torch.zeros(s["k"].shape[:2], dtype=torch.float64, device="cuda")
    q0 = 0
    for b, (t0, m, l, nq) in enumerate(zip(starts, z["new"], z["lens"], z["queries"])):
        place = torch.arange(m - nq, m, device="cuda")
        for h in range(Hkv):
            mine = (shared == h).nonzero().view(-1)
            qs, total = s["q"][q0:q0 + nq][:, mine].double(), s["lse"][q0:q0 + nq][:, mine].double()[..., None]
            near = s["seen"][b].item() + place[:, None] - s["pos"][b, h, :l].long() < window
            x = torch.exp(qs @ s["k_cache"][b, :l, h].double().T * scale - total)
            old[b, h, :l] += (x * near[:, None]).sum((0, 1))
            reach = place[:, None] - torch.arange(m, device="cuda")
            x = torch.exp(qs @ s["k"][t0:t0 + m, h].double().T * scale - total)
            new[t0:t0 + m, h] = (x * ((reach >= 0) & (reach < window))[:, None]).sum((0, 1))
        q0 += nq
    return old, new


def _exact_insert(s, z, starts):
    H, L = s["weights"].shape[1:]
    w, pos, seen = s["weights"].cpu(), s["pos"].cpu(), s["seen"].tolist()
    fresh = s["new_weights"].cpu()
    k_cache, v_cache = s["k_cache"].clone(), s["v_cache"].clone()
    w_out, pos_out, lens_out, seen_out = w.double(), pos.clone(), [], []
    slots = torch.full(fresh.shape, -1, dtype=torch.int32)
    for b, (t0, m, l) in enumerate(zip(starts, z["new"], z["lens"])):
        room, end = min(L, l + m), seen[b] + m
        lens_out.append(room)
        seen_out.append(end)
        for h in range(H):
            weight = w[b, h, :l].tolist() + fresh[t0:t0 + m, h].tolist()
            place = pos[b, h, :l].tolist() + list(range(seen[b], end))
            order = sorted(range(l + m), key=lambda i: (place[i] < end - s["recent"], 0.0 if place[i] >= end - s["recent"] else -weight[i], i))
            kept = set(order[:room])
            empty = [i for i in range(room) if i >= l or i not in kept]
            for i, to in zip((i for i in range(l, l + m) if i in kept), empty):
                w_out[b, h, to], pos_out[b, h, to], slots[t0 + i - l, h] = weight[i], place[i], to
        put = slots[t0:t0 + m].long()
        j, h = (put >= 0).nonzero(as_tuple=True)
        k_cache[b, put[j, h].cuda(), h.cuda()] = s["k"][t0 + j.cuda(), h.cuda()]
        v_cache[b, put[j, h].cuda(), h.cuda()] = s["v"][t0 + j.cuda(), h.cuda()]
    whole = lambda v: torch.tensor(v, dtype=torch.int32)                                     # noqa: E731
    return k_cache, v_cache, w_out, pos_out, whole(lens_out), whole(seen_out), slots
