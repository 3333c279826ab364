"""The operators of a bounded, shared KV cache, as cases to time and to compare.

Four operators work on the KV cache of the full-attention layers in a verify
or decode step: attention with a sliding window and visible first tokens,
attention of a batch over one shared prefix, the accumulation of attention
weights per cached key, and the eviction by those weights that also appends
the accepted draft tokens.  ``listed()`` gives named cases, ``draw(rng)``
others of the same ranges; ``prepare`` makes a case's inputs on the GPU,
``run`` makes one pass, in plain torch operations (``own`` false) or through
the library's calls (``own`` true), ``exact`` gives the same in 64 bits and
``work`` the bytes and operations that a pass cannot do without.
"""
import math
import random

import numpy as np
import torch

own = False

# Sizes: "27b" is this repository's attention workload (16 full-attention
# layers, 24 query heads over 4 KV heads of dimension 256, trees of 22 nodes,
# 1 or 5 requests); the others are generic head layouts.  ctx_lo .. ctx_hi are
# the requests' context lengths, spread evenly; T is the cache's capacity.
_ATTN27B = {"Hq": 24, "Hkv": 4, "dh": 256, "dtype": "bf16"}


def listed():
    return [
        # one layer's decode step of one request: the shortest call a decoder makes
        {"name": "window_decode_1layer", "op": "window", "L": 1, "Bq": 1, "N": 1, **_ATTN27B,
         "T": 2048, "ctx_lo": 2000, "ctx_hi": 2000, "window": 512, "n_sink": 4, "path": 1},
        # the budget-22 verify of one request, all layers, a window of 1024 over 4096 keys
        {"name": "window_tree27b", "op": "window", "L": 16, "Bq": 1, "N": 22, **_ATTN27B,
         "T": 4096, "ctx_lo": 4096, "ctx_hi": 4096, "window": 1024, "n_sink": 4, "path": 6},
        # five requests served together, a long window over ragged contexts
        {"name": "window_serve27b", "op": "window", "L": 16, "Bq": 5, "N": 22, **_ATTN27B,
         "T": 8192, "ctx_lo": 4097, "ctx_hi": 8192, "window": 4096, "n_sink": 16, "path": 6},
        # plain decode of a wide batch over long caches (no window), 16-bit floats
        {"name": "window_off_decode", "op": "window", "L": 4, "Bq": 16, "N": 1, "Hq": 32, "Hkv": 8,
         "dh": 128, "dtype": "f16", "T": 16384, "ctx_lo": 8001, "ctx_hi": 16384, "window": 0,
         "n_sink": 0, "path": 1},
        # one layer's decode step of five chats that share a system prompt
        {"name": "prefix_decode_1layer", "op": "prefix", "L": 1, "Bq": 5, "N": 1, **_ATTN27B,
         "P": 1000, "T": 256, "ctx_lo": 37, "ctx_hi": 211, "path": 1},
        # the five requests' budget-22 verify over a shared prompt of 4096 tokens
        {"name": "prefix_serve27b", "op": "prefix", "L": 16, "Bq": 5, "N": 22, **_ATTN27B,
         "P": 4096, "T": 1024, "ctx_lo": 501, "ctx_hi": 1024, "path": 6},
        # 64 samples drawn from one long document
        {"name": "prefix_samples64", "op": "prefix", "L": 2, "Bq": 64, "N": 1, "Hq": 16, "Hkv": 2,
         "dh": 128, "dtype": "f16", "P": 32001, "T": 512, "ctx_lo": 1, "ctx_hi": 512, "path": 1},
        # weights of one decoded token, one layer
        {"name": "mass_decode_1layer", "op": "mass", "L": 1, "Bq": 1, "N": 1, **_ATTN27B,
         "T": 4096, "ctx_lo": 3001, "ctx_hi": 3001, "path": 1},
        # weights of the accepted paths of five budget-22 trees, all layers
        {"name": "mass_serve27b", "op": "mass", "L": 16, "Bq": 5, "N": 22, **_ATTN27B,
         "T": 8192, "ctx_lo": 4097, "ctx_hi": 8192, "path": 6},
        # long accepted paths: more query rows than one tile holds
        {"name": "mass_longpath", "op": "mass", "L": 4, "Bq": 8, "N": 64, "Hq": 32, "Hkv": 8,
         "dh": 128, "dtype": "f16", "T": 4096, "ctx_lo": 2047, "ctx_hi": 4096, "path": 40},
        # a full cache that takes each step's accepted tokens and drops as many
        {"name": "evict_steady27b", "op": "evict", "L": 16, "Bq": 1, "N": 22, **_ATTN27B,
         "T": 4096, "ctx_lo": 4096, "ctx_hi": 4096, "path": 6, "budget": 4096, "n_sink": 4,
         "n_recent": 256},
        # prompts cut down to an eighth after prefill
        {"name": "evict_prompt", "op": "evict", "L": 8, "Bq": 5, "N": 1, **_ATTN27B,
         "T": 16384, "ctx_lo": 10001, "ctx_hi": 16384, "path": 1, "budget": 2048, "n_sink": 4,
         "n_recent": 512},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "prefix", "mass", "evict"])
    c = {"op": op, "L": _log_int(rng, 1, 16), "Bq": _log_int(rng, 1, 64), "N": _log_int(rng, 1, 64),
         "Hkv": rng.randint(1, 8), "dh": rng.choice([64, 128, 256]),
         "dtype": rng.choice(["bf16", "f16"])}
    c["Hq"] = c["Hkv"] * rng.randint(1, 8)
    c["path"] = _log_int(rng, 1, c["N"])
    c["ctx_hi"] = _log_int(rng, 1, 16384)
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    c["T"] = c["ctx_hi"] + rng.choice([0, 1, rng.randint(2, 300)])
    if op == "window":
        c["window"] = rng.choice([0, _log_int(rng, 16, 8192)])
        c["n_sink"] = rng.choice([0, rng.randint(1, 64)])
    if op == "prefix":
        c["P"] = _log_int(rng, 1, 32768)
        c["ctx_hi"], c["T"] = min(c["ctx_hi"], 2048), min(c["T"], 2100)
        c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
    # no more than the largest listed case costs, and room for the plain form
    limit = max(_cost(k) for k in listed())
    while _cost(c) > limit or _plain_bytes(c) > 12e9:
        key = max(("L", "Bq", "ctx_hi"), key=lambda k: c[k] / {"L": 4, "Bq": 4, "ctx_hi": 2048}[k])
        if c[key] == 1:
            key = "N" if c["N"] > 1 else "P"
        c[key] = max(1, c[key] // 2)
        c["ctx_lo"], c["path"] = min(c["ctx_lo"], c["ctx_hi"]), min(c["path"], c["N"])
        c["T"] = c["ctx_hi"] + (c["T"] & 1)
    if op == "evict":
        c["budget"] = rng.randint(min(c["T"], c["N"] + 64), c["T"])
        c["n_sink"] = rng.randint(0, c["budget"] // 8)
        c["n_recent"] = rng.randint(0, c["budget"] // 2)
    return c


def _cost(case):
    w = work(dict(case, budget=case.get("budget", case["T"] // 2)))
    return max(w["bytes"], w["flops"] / 50)


def _plain_bytes(case):
    keys = case["T"] + case["N"] + case.get("P", 0)
    rows = case["L"] * case["Bq"] * case["N"] * case["Hq"]
    return 16 * rows * keys + 16 * case["L"] * case["Bq"] * keys * case["Hkv"] * case["dh"]


def _contexts(case):
    lo, hi, n = case["ctx_lo"], case["ctx_hi"], case["Bq"]
    return [hi if n == 1 else lo + (hi - lo) * b // (n - 1) for b in range(n)]


def work(case):
    """Visible keys and values once (the shared prefix once for all), queries
    in, outputs out; two products of 2 dh operations per query row and visible
    key (one for the weights alone).  The tree's own keys count one per row."""
    L, Bq, N, Hq, Hkv, dh = (case[k] for k in ("L", "Bq", "N", "Hq", "Hkv", "dh"))
    ctx, rows = _contexts(case), N * Hq
    if case["op"] in ("window", "prefix"):
        W, S = case.get("window", 0), case.get("n_sink", 0)
        lo = [max(0, t - W + 1) if W else 0 for t in ctx]
        seen = [t - a + min(S, a) for t, a in zip(ctx, lo)]
        P = case.get("P", 0)
        keys = sum(seen) + Bq * N + P
        return {"bytes": L * (keys * Hkv * dh * 4 + Bq * rows * (dh * 4 + 4)),
                "flops": 4 * L * rows * dh * (sum(seen) + Bq * (1 + P))}
    if case["op"] == "mass":
        path = case["path"]
        return {"bytes": L * (sum(ctx) * Hkv * (dh * 2 + 8) + Bq * path * (Hkv * dh * 2 + Hq * (dh * 2 + 4))
                              + Bq * N * Hkv * 4),
                "flops": 2 * L * path * Hq * dh * (sum(ctx) + Bq)}
    # eviction: every score and position; of the entries that stay, those past
    # the budget's end move (an even spread of the survivors over the cache)
    moved = score_bytes = 0
    for t in ctx:
        n = t + case["path"]
        score_bytes += 8 * t + 4 * case["path"]
        kept = min(n, case["budget"])
        moved += kept - kept * min(t, kept) // n if n > case["budget"] else case["path"]
    return {"bytes": L * Hkv * (score_bytes + moved * (dh * 8 + 8)), "flops": 0}


# ---- inputs -----------------------------------------------------------------

def _tree(rng, N, path):
    """A random tree, node 0 its root, with a root-to-node path of `path` nodes."""
    chain = [0] + sorted(rng.sample(range(1, N), path - 1))
    parent = [-1] + [rng.randrange(i) for i in range(1, N)]
    for up, node in zip(chain, chain[1:]):
        parent[node] = up
    return parent, chain[-1]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    L, Bq, N, Hq, Hkv, dh, T = (case[k] for k in ("L", "Bq", "N", "Hq", "Hkv", "dh", "T"))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    trees = [_tree(rng, N, case["path"]) for _ in range(Bq)]
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"case": dict(case), "scale": dh ** -0.5,
         "ctx_len": torch.tensor(_contexts(case), **i32),
         "parent": torch.tensor([t[0] for t in trees], **i32),
         "accepted": torch.tensor([t[1] for t in trees], **i32),
         # queries twice as wide as keys: weights that gather on some keys
         "q": normal(L, Bq, N, Hq, dh) * 2,
         "k_cache": normal(L, Bq, T, Hkv, dh), "v_cache": normal(L, Bq, T, Hkv, dh),
         "k_tree": normal(L, Bq, N, Hkv, dh), "v_tree": normal(L, Bq, N, Hkv, dh)}
    if case["op"] == "prefix":
        s["k_prefix"] = normal(L, case["P"], Hkv, dh)
        s["v_prefix"] = normal(L, case["P"], Hkv, dh)
    if case["op"] in ("window", "prefix"):
        s["o"] = torch.empty(L, Bq, N, Hq, dh, device="cuda", dtype=dt)
        s["lse"] = torch.empty(L, Bq, N, Hq, device="cuda")
    if case["op"] in ("mass", "evict"):
        # weights gathered over earlier steps: heavy-tailed, as attention's are
        s["score"] = torch.empty(L, Bq, Hkv, T, device="cuda").log_normal_(0.0, 2.0, generator=g)
        s["score_tree"] = torch.empty(L, Bq, Hkv, N, device="cuda").log_normal_(0.0, 2.0, generator=g)
    if case["op"] == "mass":
        s["lse"] = _logits(s).logsumexp(-1).view(L, Bq, Hkv, N, Hq // Hkv)
        s["lse"] = s["lse"].transpose(2, 3).reshape(L, Bq, N, Hq).contiguous()
    if case["op"] == "evict":
        # absolute positions: three tokens seen for every two still cached
        t = torch.arange(T, device="cuda")
        s["pos"] = (t + t // 2).to(torch.int32).expand(L, Bq, Hkv, T).contiguous()
        s["seen"] = s["ctx_len"] + s["ctx_len"] // 2
        s["ctx_out"], s["seen_out"] = torch.empty(Bq, **i32), torch.empty(Bq, **i32)
        s["steady"] = case["ctx_lo"] == case["budget"]
        s["filled"] = {k: s[k][..., :case["budget"]].clone() for k in ("score", "pos")}
    if own:
        from tree_verify_linear_gb300 import lbx
        s["lbx"] = lbx
        s["cfg"] = lbx.make_attn_cfg(
            L=L, Bq=Bq, N=N, Hq=Hq, Hkv=Hkv, dh=dh, T=T, P=case.get("P", 0),
            window=case.get("window", 0), n_sink=case.get("n_sink", 0),
            dtype=lbx.LBX_BF16 if case["dtype"] == "bf16" else lbx.LBX_F16, scale=s["scale"])
        if case["op"] in ("window", "prefix"):
            s["workspace"] = lbx.new_cache_attn_workspace(s["cfg"])
    return s


# ---- the plain forms ----------------------------------------------------------

def _ancestors(parent):
    """[Bq][N][N]: node m is node n or one of its ancestors; [Bq][N] depths."""
    N = parent.shape[1]
    step = torch.eye(N, device="cuda", dtype=torch.float64) + (
        parent[:, :, None] == torch.arange(N, device="cuda")).double()
    anc = torch.linalg.matrix_power(step, N) > 0
    return anc, anc.sum(-1) - 1


def _grouped(q, Hkv):
    """Query rows (node, head of the group) of each KV head, in 32 bits."""
    L, Bq, N, Hq, dh = q.shape
    return q.float().view(L, Bq, N, Hkv, Hq // Hkv, dh).transpose(2, 3).reshape(
        L, Bq, Hkv, N * (Hq // Hkv), dh)


def _visible(s):
    """[Bq][N][T + N]: which cached keys and tree nodes each node's query sees."""
    c = s["case"]
    N, T, W, S = c["N"], c["T"], c.get("window", 0), c.get("n_sink", 0)
    anc, depth = _ancestors(s["parent"])
    ctx = s["ctx_len"].long()
    at = ctx[:, None] + depth  # positions of the nodes
    j = torch.arange(T, device="cuda")
    old = (j < ctx[:, None])[:, None, :].expand(-1, N, -1)
    new = anc
    if W > 0:
        old = old & ((at[:, :, None] - j < W) | (j < S))
        new = new & ((depth[:, :, None] - depth[:, None, :] < W) | (at[:, None, :] < S))
    return torch.cat([old, new], -1)


def _logits(s):
    """Scaled, masked scores [L][Bq][Hkv][N G][T + N] of cache and tree."""
    c = s["case"]
    q = _grouped(s["q"], c["Hkv"])
    k = torch.cat([s["k_cache"], s["k_tree"]], 2).float().permute(0, 1, 3, 4, 2)
    x = (q @ k) * s["scale"]
    seen = _visible(s).repeat_interleave(c["Hq"] // c["Hkv"], 1)[None, :, None]
    return torch.where(seen, x, -math.inf)


def _plain_attention(s):
    c = s["case"]
    L, Bq, N, Hq, Hkv, dh, T, P = (c.get(k, 0) for k in ("L", "Bq", "N", "Hq", "Hkv", "dh", "T", "P"))
    G = Hq // Hkv
    x = _logits(s)
    # values that no query sees may hold anything: they take no part
    live = (torch.arange(T, device="cuda") < s["ctx_len"][:, None])[None, :, :, None, None]
    v = torch.cat([torch.where(live, s["v_cache"], 0), s["v_tree"]], 2).float().transpose(2, 3)
    m = x.amax(-1, keepdim=True)
    if P:
        q = _grouped(s["q"], Hkv).transpose(1, 2).reshape(L, Hkv, Bq * N * G, dh)
        xp = (q @ s["k_prefix"].float().permute(0, 2, 3, 1)) * s["scale"]
        mp = xp.amax(-1, keepdim=True).view(L, Hkv, Bq, N * G, 1).transpose(1, 2)
        m = torch.maximum(m, mp)
    e = torch.exp(x - m)
    total, o = e.sum(-1, keepdim=True), e @ v
    if P:
        e = torch.exp(xp - m.transpose(1, 2).reshape(L, Hkv, Bq * N * G, 1))
        op = e @ s["v_prefix"].float().transpose(1, 2)
        total = total + e.sum(-1, keepdim=True).view(L, Hkv, Bq, N * G, 1).transpose(1, 2)
        o = o + op.view(L, Hkv, Bq, N * G, dh).transpose(1, 2)
    o = (o / total).view(L, Bq, Hkv, N, G, dh).transpose(2, 3).reshape(L, Bq, N, Hq, dh)
    lse = (m + torch.log(total)).view(L, Bq, Hkv, N, G).transpose(2, 3).reshape(L, Bq, N, Hq)
    return {"o": o.to(s["q"].dtype), "lse": lse}


def _on_path(s):
    """[Bq][N]: the nodes of the path from the root to the accepted node."""
    anc, depth = _ancestors(s["parent"])
    at = s["accepted"].long()[:, None, None].expand(-1, 1, anc.shape[-1])
    return anc.gather(1, at)[:, 0], depth


def _plain_mass(s):
    c = s["case"]
    L, Bq, N, Hq, Hkv, T = (c[k] for k in ("L", "Bq", "N", "Hq", "Hkv", "T"))
    G = Hq // Hkv
    lse = s["lse"].view(L, Bq, N, Hkv, G).transpose(2, 3).reshape(L, Bq, Hkv, N * G, 1)
    w = torch.exp(_logits(s) - lse)
    on = _on_path(s)[0]
    w = torch.where(on.repeat_interleave(G, 1)[None, :, None, :, None], w, 0).sum(-2)
    s["score"].add_(w[..., :T])
    s["score_tree"].copy_(torch.where(on[None, :, None], w[..., T:], 0))
    return {"score": s["score"], "score_tree": s["score_tree"]}


def _plain_evict(s):
    c = s["case"]
    L, Bq, N, Hkv, dh, T, budget = (c[k] for k in ("L", "Bq", "N", "Hkv", "dh", "T", "budget"))
    on, depth = _on_path(s)
    ctx, path = s["ctx_len"].long(), on.sum(-1)
    seen = s["seen"].long() + path
    # the accepted path's nodes in order of depth, behind the cache's entries
    node = torch.where(on, depth, N + depth).argsort(dim=-1, stable=True)
    at = node[None, :, None].expand(L, -1, Hkv, -1)
    score = torch.cat([s["score"], s["score_tree"].gather(-1, at)], -1)
    step = torch.arange(N, device="cuda")
    pos = torch.cat([s["pos"], (s["seen"][:, None] + step)[None, :, None].expand(L, -1, Hkv, -1)], -1)
    t = torch.arange(T, device="cuda")
    real = torch.cat([t < ctx[:, None], step < path[:, None]], -1)[None, :, None]
    safe = (pos < c["n_sink"]) | (pos >= (seen - c["n_recent"])[:, None, None])
    rank = torch.where(real, torch.where(safe, math.inf, score), -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    n = (ctx + path).clamp(max=budget)
    keep = torch.zeros_like(rank, dtype=torch.bool).scatter_(
        -1, order, (torch.arange(T + N, device="cuda") < n[:, None])[None, :, None].expand_as(rank))
    # kept entries past the new end fill the free slots before it, in order
    slot = torch.arange(T + N, device="cuda")
    low = (slot < torch.minimum(ctx, n)[:, None])[None, :, None]
    free = (slot < n[:, None])[None, :, None] & ~(keep & low)
    mover = keep & ~low
    src, dst = mover.nonzero(), free.nonzero()
    l, b, h, a = src.unbind(-1)
    z = dst[:, 3]
    cached = a < T
    a0, a1 = a.clamp(max=T - 1), node[b, (a - T).clamp(min=0)]
    for_k = torch.where(cached[:, None], s["k_cache"][l, b, a0, h], s["k_tree"][l, b, a1, h])
    for_v = torch.where(cached[:, None], s["v_cache"][l, b, a0, h], s["v_tree"][l, b, a1, h])
    s["k_cache"][l, b, z, h] = for_k
    s["v_cache"][l, b, z, h] = for_v
    s["score"][l, b, h, z] = score[l, b, h, a]
    s["pos"][l, b, h, z] = pos[l, b, h, a].to(torch.int32)
    s["ctx_out"].copy_(n)
    s["seen_out"].copy_(seen)


def run(s):
    c = s["case"]
    if c["op"] == "evict" and not s["steady"]:
        # a new prompt's weights and positions, where the last eviction put its own
        s["score"][..., :c["budget"]].copy_(s["filled"]["score"])
        s["pos"][..., :c["budget"]].copy_(s["filled"]["pos"])
    if not own:
        if c["op"] in ("window", "prefix"):
            return _plain_attention(s)
        if c["op"] == "mass":
            return _plain_mass(s)
        _plain_evict(s)
    elif c["op"] == "window":
        s["lbx"].lbx_window_attention(
            s["cfg"], s["ctx_len"], s["parent"], s["q"], s["k_cache"], s["v_cache"], s["k_tree"],
            s["v_tree"], s["o"], s["workspace"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    elif c["op"] == "prefix":
        s["lbx"].lbx_prefix_attention(
            s["cfg"], s["ctx_len"], s["parent"], s["q"], s["k_prefix"], s["v_prefix"],
            s["k_cache"], s["v_cache"], s["k_tree"], s["v_tree"], s["o"], s["workspace"],
            lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    elif c["op"] == "mass":
        s["lbx"].lbx_attention_mass(
            s["cfg"], s["ctx_len"], s["parent"], s["accepted"], s["q"], s["lse"], s["k_cache"],
            s["k_tree"], s["score"], s["score_tree"])
        return {"score": s["score"], "score_tree": s["score_tree"]}
    else:
        s["lbx"].lbx_cache_evict(
            s["cfg"], c["budget"], c["n_recent"], s["ctx_len"], s["seen"], s["parent"],
            s["accepted"], s["k_tree"], s["v_tree"], s["score_tree"], s["k_cache"], s["v_cache"],
            s["score"], s["pos"], s["ctx_out"], s["seen_out"])
    out = {k: s[k] for k in ("k_cache", "v_cache", "score", "pos", "ctx_out", "seen_out")}
    if s["steady"]:
        # a full cache's next step goes on from this one's lengths
        s["ctx_len"], s["ctx_out"] = s["ctx_out"], s["ctx_len"]
        s["seen"], s["seen_out"] = s["seen_out"], s["seen"]
    return out


# ---- the definitions, in 64 bits -----------------------------------------------

def _up(parent, n):
    """Node n's root-to-node path."""
    path = []
    while n >= 0:
        path.append(n)
        n = parent[n]
    return path[::-1]


def exact(case, seed):
    s = prepare(case, seed)
    parent, ctx = s["parent"].tolist(), s["ctx_len"].tolist()
    if case["op"] == "evict":
        return _exact_evict(case, s, parent, ctx)
    L, Bq, N, Hq, Hkv, dh = (case[k] for k in ("L", "Bq", "N", "Hq", "Hkv", "dh"))
    G, W, S, P = Hq // Hkv, case.get("window", 0), case.get("n_sink", 0), case.get("P", 0)
    f64 = {"dtype": torch.float64, "device": "cuda"}
    o, lse = torch.zeros(L, Bq, N, Hq, dh, **f64), torch.zeros(L, Bq, N, Hq, **f64)
    if case["op"] == "mass":
        score, score_tree = s["score"].double(), torch.zeros(L, Bq, Hkv, N, **f64)
        accepted = s["accepted"].tolist()
    for b in range(Bq):
        t = ctx[b]
        allowed = np.zeros((N, t + N), dtype=bool)
        for n in range(N):
            up = _up(parent[b], n)
            p = t + len(up) - 1
            first = max(0, p - W + 1) if W else 0
            allowed[n, min(first, t):t] = True
            allowed[n, :min(S, t)] = True
            for d, m in enumerate(up):
                allowed[n, t + m] = t + d >= first or t + d < S
        hide = torch.from_numpy(~allowed).cuda()
        for l in range(L):
            for h in range(Hkv):
                q = s["q"][l, b, :, h * G:(h + 1) * G].double()
                k = torch.cat([s["k_cache"][l, b, :t, h], s["k_tree"][l, b, :, h]]).double()
                x = torch.einsum("ngd,td->ngt", q, k) * s["scale"]
                x.masked_fill_(hide[:, None], -math.inf)
                if case["op"] == "mass":
                    up = _up(parent[b], accepted[b])
                    lb = s["lse"][l, b, up, h * G:(h + 1) * G].double()
                    w = torch.exp(x[up] - lb[..., None]).sum((0, 1))
                    score[l, b, h, :t] += w[:t]
                    score_tree[l, b, h, up] = w[t:][up]
                    continue
                v = torch.cat([s["v_cache"][l, b, :t, h], s["v_tree"][l, b, :, h]]).double()
                if P:
                    x = torch.cat([torch.einsum("ngd,td->ngt", q, s["k_prefix"][l, :, h].double())
                                   * s["scale"], x], -1)
                    v = torch.cat([s["v_prefix"][l, :, h].double(), v])
                z = torch.logsumexp(x, -1)
                lse[l, b, :, h * G:(h + 1) * G] = z
                o[l, b, :, h * G:(h + 1) * G] = torch.einsum(
                    "ngt,td->ngd", torch.exp(x - z[..., None]), v)
    if case["op"] == "mass":
        return {"score": score, "score_tree": score_tree}
    return {"o": o, "lse": lse}


def _exact_evict(case, s, parent, ctx):
    """One (layer, request, KV head) after the other, on the host's indexes."""
    score, tree = s["score"].cpu().numpy(), s["score_tree"].cpu().numpy()
    pos, seen = s["pos"].cpu().numpy(), s["seen"].tolist()
    ctx_out, seen_out = list(ctx), list(seen)
    for b in range(case["Bq"]):
        t, up = ctx[b], _up(parent[b], s["accepted"].tolist()[b])
        n, end = t + len(up), seen[b] + len(up)
        size = min(n, case["budget"])
        ctx_out[b], seen_out[b] = size, end
        for l in range(case["L"]):
            for h in range(case["Hkv"]):
                p = np.concatenate([pos[l, b, h, :t], seen[b] + np.arange(len(up))])
                w = np.concatenate([score[l, b, h, :t], tree[l, b, h, up]])
                safe = (p < case["n_sink"]) | (p >= end - case["n_recent"])
                rank = np.where(safe, np.inf, w.astype(np.float64))
                best = np.sort(np.argsort(-rank, kind="stable")[:size])
                low = min(t, size)
                movers = best[best >= low]
                if not len(movers):
                    continue
                holes = np.setdiff1d(np.arange(size), best[best < low])
                score[l, b, h, holes], pos[l, b, h, holes] = w[movers], p[movers]
                held, fresh = movers[movers < t], movers[movers >= t] - t
                to = torch.from_numpy(holes).cuda()
                for cache, new in (("k_cache", "k_tree"), ("v_cache", "v_tree")):
                    rows = [s[cache][l, b, torch.from_numpy(held).cuda(), h],
                            s[new][l, b, [up[i] for i in fresh], h]]
                    s[cache][l, b, to, h] = torch.cat(rows)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "score": torch.from_numpy(score).cuda(),
            "pos": torch.from_numpy(pos).cuda(), "ctx_out": torch.tensor(ctx_out, **i32),
            "seen_out": torch.tensor(seen_out, **i32)}
