"""The operators of a paged KV cache, as cases to time and to compare.

Four operators serve requests whose keys and values lie in pages of one pool:
the block tables and slot maps of a step from the requests' lengths; the norms
of queries and keys per head with the position rotation, which also puts keys
and values into their pages; the attention of each request's new tokens (a
prompt's chunk, a draft tree, a single token) over its pages; and the commit of
a verified path, which closes the gaps that rejected draft tokens left.
``listed()`` gives named cases, ``draw(rng)`` others of the same ranges;
``prepare`` makes a case's inputs on the GPU, ``run`` makes one pass, in plain
torch operations (``own`` false) or through the library's calls (``own`` true),
``exact`` gives the same in 64 bits and ``work`` the bytes and operations that a
pass cannot do without.
"""
import math
import random

import numpy as np
import torch

own = False

# "27b" is this repository's attention workload (16 full-attention layers, 24
# query heads over 4 KV heads of dimension 256, trees of 22 nodes, 1 or 5
# requests); the others are generic head layouts.  Requests have ctx_lo ..
# ctx_hi cached positions and n_lo .. n_hi new tokens, both spread evenly over
# the batch, the longest context with the fewest new tokens; pad rows follow.
_27B = {"Hq": 24, "Hkv": 4, "dh": 256, "dtype": "bf16"}


def listed():
    return [
        # a decode step of a wide batch: a page runs full here and there, some requests ended
        {"name": "tables_decode", "op": "tables", "Bq": 256, "ctx_lo": 100, "ctx_hi": 16000,
         "n_lo": 1, "n_hi": 1, "pad": 0, "page": 64, "done": 8},
        # a step that takes in long prompts beside running requests, small pages
        {"name": "tables_prompts", "op": "tables", "Bq": 64, "ctx_lo": 0, "ctx_hi": 9000,
         "n_lo": 1, "n_hi": 4095, "pad": 77, "page": 16, "done": 3},
        # one layer's decode step of five requests, a quarter of the dimensions turned
        {"name": "rope_decode_1layer", "op": "rope", "L": 1, "Bq": 5, **_27B, "ctx_lo": 700,
         "ctx_hi": 8191, "n_lo": 1, "n_hi": 1, "pad": 0, "page": 64, "rot": 64, "axes": 1,
         "pairing": "halves", "base": 1e7},
        # one layer of a step that reads prompts in chunks
        {"name": "rope_prompt27b", "op": "rope", "L": 1, "Bq": 4, **_27B, "ctx_lo": 0,
         "ctx_hi": 30000, "n_lo": 1025, "n_hi": 3001, "pad": 0, "page": 64, "rot": 64, "axes": 1,
         "pairing": "halves", "base": 1e7},
        # tokens of video frames: time, height and width turn a part of the pairs each
        {"name": "rope_video", "op": "rope", "L": 1, "Bq": 2, "Hq": 32, "Hkv": 8, "dh": 128,
         "dtype": "f16", "ctx_lo": 33, "ctx_hi": 4001, "n_lo": 6007, "n_hi": 9999, "pad": 5,
         "page": 16, "rot": 128, "axes": 3, "pairing": "adjacent", "base": 1e6},
        # one layer's decode step of one request: the shortest call a decoder makes
        {"name": "attend_decode_1layer", "op": "attend", "L": 1, "Bq": 1, **_27B, "ctx_lo": 2000,
         "ctx_hi": 2000, "n_lo": 1, "n_hi": 1, "pad": 0, "page": 64, "tree": False},
        # the budget-22 verify of five requests, all layers
        {"name": "attend_tree27b", "op": "attend", "L": 16, "Bq": 5, **_27B, "ctx_lo": 2049,
         "ctx_hi": 4096, "n_lo": 22, "n_hi": 22, "pad": 0, "page": 64, "tree": True},
        # plain decode of a wide batch over long caches, 16-bit floats, small pages
        {"name": "attend_decode_long", "op": "attend", "L": 4, "Bq": 16, "Hq": 32, "Hkv": 8,
         "dh": 128, "dtype": "f16", "ctx_lo": 8001, "ctx_hi": 16384, "n_lo": 1, "n_hi": 1,
         "pad": 0, "page": 16, "tree": False},
        # one layer over a chunk of a long prompt
        {"name": "attend_chunk27b", "op": "attend", "L": 1, "Bq": 1, **_27B, "ctx_lo": 6144,
         "ctx_hi": 6144, "n_lo": 2048, "n_hi": 2048, "pad": 0, "page": 64, "tree": False},
        # whole prompts of odd lengths, nothing cached
        {"name": "attend_prompts", "op": "attend", "L": 1, "Bq": 6, "Hq": 32, "Hkv": 8,
         "dh": 128, "dtype": "bf16", "ctx_lo": 0, "ctx_hi": 0, "n_lo": 501, "n_hi": 6001,
         "pad": 9, "page": 32, "tree": False},
        # the accepted paths of five budget-22 trees, all layers
        {"name": "commit_serve27b", "op": "commit", "L": 16, "Bq": 5, **_27B, "ctx_lo": 2049,
         "ctx_hi": 4096, "n_lo": 22, "n_hi": 22, "pad": 0, "page": 64, "path": 6},
        # long accepted paths of a wide batch, small pages
        {"name": "commit_longpath", "op": "commit", "L": 16, "Bq": 64, "Hq": 32, "Hkv": 8,
         "dh": 128, "dtype": "f16", "ctx_lo": 15, "ctx_hi": 1000, "n_lo": 64, "n_hi": 64,
         "pad": 0, "page": 16, "path": 40},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "attend", "attend", "commit"])
    c = {"op": op, "Bq": _log_int(rng, 1, 64), "page": rng.choice([16, 32, 64, 128, 256]),
         "pad": rng.choice([0, rng.randint(1, 40)])}
    c["ctx_hi"] = _log_int(rng, 1, 16384)
    c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
    c["n_hi"] = _log_int(rng, 1, 4096)
    c["n_lo"] = rng.randint(1, c["n_hi"])
    if op == "tables":
        c["Bq"] = _log_int(rng, 1, 512)
        c["done"] = rng.randint(0, c["Bq"] // 8)
    else:
        c.update(L=_log_int(rng, 1, 16), Hkv=rng.randint(1, 8), dh=rng.choice([64, 128, 256]),
                 dtype=rng.choice(["bf16", "f16"]))
        c["Hq"] = c["Hkv"] * rng.randint(1, 8)
    if op == "rope":
        c["axes"] = rng.choice([1, 1, 3])
        c["rot"] = 2 * rng.randint(c["axes"], c["dh"] // 2)
        c["pairing"] = rng.choice(["halves", "adjacent"])
        c["base"] = 10.0 ** rng.uniform(4, 7)
    if op == "attend":
        c["tree"] = rng.choice([True, False, False])
    if op == "commit" or c.get("tree"):
        c["n_hi"] = _log_int(rng, 1, 64)
        c["n_lo"] = rng.randint(1, c["n_hi"])
    if op == "commit":
        c["path"] = _log_int(rng, 1, c["n_lo"])
    # no more than the largest listed case costs, and room for the plain form
    limit = max(_cost(k) for k in listed())
    room = {"L": 4, "Bq": 4, "ctx_hi": 2048, "n_hi": 1024}
    while _cost(c) > limit or _plain_bytes(c) > 12e9:
        key = max((k for k in room if k in c), key=lambda k: c[k] / room[k])
        c[key] = max(1, c[key] // 2)
        c["ctx_lo"], c["n_lo"] = min(c["ctx_lo"], c["ctx_hi"]), min(c["n_lo"], c["n_hi"])
        if "path" in c:
            c["path"] = min(c["path"], c["n_lo"])
    return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 250)


def _plain_bytes(case):
    if case["op"] == "tables":
        return 0
    ctx, new = _lengths(case)
    pool = 12 * case["L"] * case["Hkv"] * case["dh"] * (sum(ctx) + sum(new) + case["Bq"] * case["page"])
    rows = 24 * case["L"] * sum(new) * (case["Hq"] + 2 * case["Hkv"]) * case["dh"]
    scores = max(16 * case["L"] * n * case["Hq"] * (t + n) for t, n in zip(ctx, new))
    return pool + rows + (scores if case["op"] == "attend" else 0)


def _lengths(case):
    """Cached positions and new tokens of each request."""
    B = case["Bq"]

    def spread(lo, hi, b):
        return hi if B == 1 else lo + (hi - lo) * b // (B - 1)

    return ([spread(case["ctx_lo"], case["ctx_hi"], b) for b in range(B)],
            [spread(case["n_lo"], case["n_hi"], B - 1 - b) for b in range(B)])


def work(case):
    """Tables: the lengths in, the tables' new entries and the maps out.  Rope:
    the projections in, queries, keys and values out.  Attention: visible keys
    and values once per layer, queries in, outputs out; two products of 2 dh
    operations per query row and visible key (a tree's own keys count one per
    row).  Commit: keys and values of a path behind its root, in and out."""
    ctx, new = _lengths(case)
    M, B = sum(new), case["Bq"]
    if case["op"] == "tables":
        fresh = sum(-(-(t + n) // case["page"]) - -(-t // case["page"]) for t, n in zip(ctx, new))
        return {"bytes": 8 * (M + case["pad"]) + 20 * B + 8 * fresh, "flops": 0}
    L, Hq, Hkv, dh = (case[k] for k in ("L", "Hq", "Hkv", "dh"))
    if case["op"] == "rope":
        return {"bytes": L * M * ((Hq + 2 * Hkv) * dh * 4 + 4) + 4 * M * case["axes"],
                "flops": 8 * L * M * (Hq + Hkv) * dh}
    if case["op"] == "commit":
        return {"bytes": 8 * L * Hkv * dh * B * (case["path"] - 1) + 12 * M, "flops": 0}
    seen = sum(n * (t + 1) if case["tree"] else n * t + n * (n + 1) // 2 for t, n in zip(ctx, new))
    return {"bytes": L * ((sum(ctx) + M) * Hkv * dh * 4 + M * Hq * (dh * 4 + 4)),
            "flops": 4 * L * Hq * dh * seen}


# ---- inputs -----------------------------------------------------------------

def _tree(rng, n, path):
    """A random tree, node 0 its root, with a root-to-node path of `path` nodes."""
    chain = [0] + sorted(rng.sample(range(1, n), path - 1))
    parent = [-1] + [rng.randrange(i) for i in range(1, n)]
    for up, node in zip(chain, chain[1:]):
        parent[node] = up
    return parent, chain[-1]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    ctx, new = _lengths(case)
    B, page, M = case["Bq"], case["page"], sum(new) + case["pad"]
    s = {"case": dict(case), "ctx": ctx, "new": new, "M": M}

    def pages_of(t):
        return -(-t // page)

    if case["op"] == "tables":
        # pages in the order that a server's traffic left; ended requests give theirs back,
        # and some hold a page that a rejected draft had needed
        held = [pages_of(t) + rng.choice([0, 0, 1]) for t in ctx]
        s["max_pages"] = max(pages_of(t + n) for t, n in zip(ctx, new)) + 3
        s["n_pages"] = sum(pages_of(t + n) + 1 for t, n in zip(ctx, new)) + 16
        for b in rng.sample(range(B), case["done"]):
            ctx[b] = new[b] = 0
            held[b] = max(held[b], 1)
        order = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32).cpu().numpy()
        table, at = np.full((B, s["max_pages"]), -1, dtype=np.int32), 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        free = np.full(s["n_pages"], -1, dtype=np.int32)
        free[:s["n_pages"] - at] = order[at:]
        s.update(ctx_len=_i32(ctx), new_len=_i32(new), held=_i32(held), n_free=_i32([s["n_pages"] - at]),
                 block_table=torch.from_numpy(table).cuda(), free_list=torch.from_numpy(free).cuda(),
                 held_out=_i32([0] * B), n_free_out=_i32([0]), start=_i32([0] * (B + 1)),
                 slot=_i32([0] * M), pos=_i32([0] * M))
        shape = {"L": 1, "Hq": 1, "Hkv": 1, "dh": 64, "dtype": "bf16"}
    else:
        shape = case
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
        L, Hq, Hkv, dh = (case[k] for k in ("L", "Hq", "Hkv", "dh"))

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda", dtype=dt)

        need = [pages_of(t + n) for t, n in zip(ctx, new)]
        s["max_pages"], s["n_pages"] = max(need), sum(need) + 1
        order = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
        s["block_table"] = torch.full((B, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, h in enumerate(need):
            s["block_table"][b, :h] = order[at:at + h]
            at += h
        s["k_pages"] = normal(L, s["n_pages"], page, Hkv, dh)
        s["v_pages"] = normal(L, s["n_pages"], page, Hkv, dh)
        s["ctx_len"] = _i32(ctx)
        start = [sum(new[:b]) for b in range(B + 1)]
        s["start"] = _i32(start)
        if case["op"] == "rope":
            # position and place of each token
            row_b = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).cuda()
            p = torch.arange(sum(new), device="cuda") - s["start"].long()[row_b] + s["ctx_len"].long()[row_b]
            slot = s["block_table"].long()[row_b, p // page] * page + p % page
            s["slot"] = torch.full((M,), -1, dtype=torch.int32, device="cuda")
            s["slot"][:len(p)] = slot.to(torch.int32)
            pos = torch.zeros((case["axes"], M), dtype=torch.int32, device="cuda")
            pos[0, :len(p)] = p.to(torch.int32)
            if case["axes"] == 3:  # frames of 40 x 36 patches
                pos[0, :len(p)] = (p // 1440).to(torch.int32)
                pos[1, :len(p)] = (p // 40 % 36).to(torch.int32)
                pos[2, :len(p)] = (p % 40).to(torch.int32)
            s["pos"] = pos
            half = case["rot"] // 2
            s["sections"] = [half] if case["axes"] == 1 else [
                half // 4, (half - half // 4) // 2, half - half // 4 - (half - half // 4) // 2]
            s["inv_freq"] = (case["base"] ** (-torch.arange(half, device="cuda", dtype=torch.float64)
                                              / half)).float()
            s["qkv"] = normal(L, M, Hq + 2 * Hkv, dh) * 2
            s["q_weight"] = 1 + torch.randn(L, dh, generator=g, device="cuda") / 4
            s["k_weight"] = 1 + torch.randn(L, dh, generator=g, device="cuda") / 4
            s["q"] = torch.zeros(L, M, Hq, dh, device="cuda", dtype=dt)
        if case["op"] == "commit" or case.get("tree"):
            trees = [_tree(rng, n, case.get("path", 1)) for n in new]
            s["parent"] = _i32([p for t in trees for p in t[0]] + [-1] * case["pad"])
            s["accepted"] = _i32([t[1] for t in trees])
            s["parents"], s["ends"] = [t[0] for t in trees], [t[1] for t in trees]
            s["ctx_out"] = _i32([0] * B)
        if case["op"] == "attend":
            # queries twice as wide as keys: weights that gather on some keys
            s["q"] = normal(L, M, Hq, dh) * 2
            s["o"] = torch.zeros(L, M, Hq, dh, device="cuda", dtype=dt)
            s["lse"] = torch.zeros(L, M, Hq, device="cuda")
    if own:
        from tree_verify_linear_gb300 import lbx
        s["lbx"] = lbx
        s["cfg"] = lbx.make_page_cfg(
            L=shape["L"], Bq=B, M=M, Hq=shape["Hq"], Hkv=shape["Hkv"], dh=shape["dh"], page=page,
            n_pages=s["n_pages"], max_pages=s["max_pages"],
            dtype=lbx.LBX_BF16 if shape["dtype"] == "bf16" else lbx.LBX_F16)
        if case["op"] == "rope":
            s["rope"] = lbx.make_rope_cfg(
                s["sections"], eps=1e-6, pairing=lbx.LBX_ROPE_HALVES if case["pairing"] == "halves"
                else lbx.LBX_ROPE_ADJACENT)
        if case["op"] == "attend":
            s["workspace"] = lbx.new_paged_workspace(s["cfg"])
    return s


# ---- the plain forms ----------------------------------------------------------

def _plain_tables(s):
    page, n_pages, width = s["case"]["page"], s["n_pages"], s["max_pages"]
    ctx, new, held = s["ctx_len"].long(), s["new_len"].long(), s["held"].long()
    table, n_free = s["block_table"], s["n_free"].long()
    want = (ctx + new + page - 1) // page
    over, lack = (held - want).clamp(min=0), (want - held).clamp(min=0)
    back, taken = over.cumsum(0) - over, lack.cumsum(0) - lack
    col = torch.arange(width, device="cuda")
    # surplus pages go behind the free ones; fresh pages come from the end
    place = torch.where((col >= want[:, None]) & (col < held[:, None]),
                        n_free + back[:, None] + col - want[:, None], n_pages)
    free = torch.cat([s["free_list"], s["free_list"][:1]]).scatter_(0, place.flatten(), table.flatten())
    s["free_list"].copy_(free[:n_pages])
    top = n_free + over.sum()
    source = (top - 1 - taken[:, None] - col + held[:, None]).clamp(0, n_pages - 1)
    fresh = (col >= held[:, None]) & (col < want[:, None])
    table.copy_(torch.where(fresh, free[source], table))
    s["held_out"].copy_(want)
    s["n_free_out"].copy_(top - lack.sum())
    end = new.cumsum(0)
    s["start"][1:] = end
    row = torch.arange(s["M"], device="cuda")
    b = torch.searchsorted(end, row, right=True).clamp(max=len(end) - 1)
    p = ctx[b] + row - (end - new)[b]
    live = row < end[-1]
    at = table[b, (p // page).clamp(max=width - 1)].long() * page + p % page
    s["slot"].copy_(torch.where(live, at, -1))
    s["pos"].copy_(torch.where(live, p, -1))


def _plain_rope(s):
    c = s["case"]
    Hq, Hkv, rot, half = c["Hq"], c["Hkv"], c["rot"], c["rot"] // 2
    live = s["slot"] >= 0
    x = s["qkv"].float()
    axis = torch.cat([torch.full((n,), a, device="cuda") for a, n in enumerate(s["sections"])])
    angle = s["pos"][axis].double().t() * s["inv_freq"].double()  # [M][half]
    cos, sin = torch.cos(angle).float()[None, :, None], torch.sin(angle).float()[None, :, None]
    out = []
    for heads, weight in ((x[:, :, :Hq], s["q_weight"]), (x[:, :, Hq:Hq + Hkv], s["k_weight"])):
        y = heads * torch.rsqrt((heads * heads).mean(-1, keepdim=True) + 1e-6) * weight[:, None, None]
        turned, rest = y[..., :rot], y[..., rot:]
        if c["pairing"] == "halves":
            a, b = turned[..., :half], turned[..., half:]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out.append(torch.cat([turned, rest], -1))
    s["q"].copy_(torch.where(live[None, :, None, None], out[0].to(s["q"].dtype), s["q"]))
    # rows without a place go to a spare row behind the pool
    n = s["n_pages"] * c["page"]
    place = torch.where(live, s["slot"], n).long()
    for pages, new in ((s["k_pages"], out[1].to(s["q"].dtype)), (s["v_pages"], s["qkv"][:, :, Hq + Hkv:])):
        flat = pages.view(c["L"], n, Hkv, c["dh"])
        spare = torch.cat([flat, flat[:, :1]], 1)
        spare[:, place] = new
        flat.copy_(spare[:, :n])


def _ancestors(parent):
    """[n][n]: node m is node n or one of its ancestors."""
    n = parent.shape[0]
    step = torch.eye(n, device="cuda", dtype=torch.float64) + (
        parent[:, None] == torch.arange(n, device="cuda")).double()
    return torch.linalg.matrix_power(step, n) > 0


def _plain_attend(s):
    c = s["case"]
    L, Hq, Hkv, dh, page = (c[k] for k in ("L", "Hq", "Hkv", "dh", "page"))
    G, at = Hq // Hkv, 0
    for b, (t, n) in enumerate(zip(s["ctx"], s["new"])):
        pages = s["block_table"][b, :-(-(t + n) // page)].long()
        k = s["k_pages"][:, pages].flatten(1, 2)[:, :t + n].float().permute(0, 2, 3, 1)
        v = s["v_pages"][:, pages].flatten(1, 2)[:, :t + n].float().transpose(1, 2)
        q = s["q"][:, at:at + n].float().view(L, n, Hkv, G, dh).permute(0, 2, 1, 3, 4)
        x = (q.reshape(L, Hkv, n * G, dh) @ k) * dh ** -0.5
        own_keys = (_ancestors(s["parent"][at:at + n]) if c["tree"] else
                    torch.ones(n, n, device="cuda", dtype=torch.bool).tril())
        x.view(L, Hkv, n, G, t + n)[..., t:].masked_fill_(~own_keys[None, None, :, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        total = e.sum(-1, keepdim=True)
        o = ((e @ v) / total).view(L, Hkv, n, G, dh).permute(0, 2, 1, 3, 4)
        s["o"][:, at:at + n] = o.reshape(L, n, Hq, dh).to(s["o"].dtype)
        lse = (m + torch.log(total)).view(L, Hkv, n, G).transpose(1, 2)
        s["lse"][:, at:at + n] = lse.reshape(L, n, Hq)
        at += n


def _plain_commit(s):
    c = s["case"]
    page, at = c["page"], 0
    for b, n in enumerate(s["new"]):
        anc = _ancestors(s["parent"][at:at + n])
        on = anc[s["accepted"][b].long()]
        # a node of the path moves to the place of its depth; the others stay
        i = torch.arange(n, device="cuda")
        depth = on.cumsum(0) - 1
        ctx = s["ctx_len"][b].long()
        src = torch.full((n,), -1, device="cuda", dtype=torch.long)
        src.scatter_reduce_(0, torch.where(on, depth, 0), torch.where(on, i, 0), "amax")
        src = torch.where(src < 0, i, src)
        src = torch.where(i == 0, 0, src)
        p = ctx + i
        place = s["block_table"][b, p // page].long() * page + p % page
        for pages in (s["k_pages"], s["v_pages"]):
            flat = pages.view(c["L"], -1, c["Hkv"], c["dh"])
            flat[:, place] = flat[:, place[src]]
        s["ctx_out"][b] = (ctx + on.sum()).to(torch.int32)
        at += n


def run(s):
    op, lbx, cfg = s["case"]["op"], s.get("lbx"), s.get("cfg")
    if not own:
        {"tables": _plain_tables, "rope": _plain_rope, "attend": _plain_attend,
         "commit": _plain_commit}[op](s)
    elif op == "tables":
        lbx.lbx_page_tables(cfg, s["ctx_len"], s["new_len"], s["held"], s["n_free"], s["block_table"],
                            s["free_list"], s["held_out"], s["n_free_out"], s["start"], s["slot"],
                            s["pos"])
    elif op == "rope":
        lbx.lbx_qk_norm_rope(cfg, s["rope"], s["qkv"], s["inv_freq"], s["pos"], s["slot"], s["q"],
                             s["k_pages"], s["v_pages"], q_weight=s["q_weight"],
                             k_weight=s["k_weight"])
    elif op == "attend":
        lbx.lbx_paged_attention(cfg, s["start"], s["ctx_len"], s["block_table"], s["q"], s["k_pages"],
                                s["v_pages"], s["o"], s["workspace"],
                                parent=s["parent"] if s["case"]["tree"] else None, lse=s["lse"])
    else:
        lbx.lbx_page_commit(cfg, s["start"], s["ctx_len"], s["block_table"], s["parent"],
                            s["accepted"], s["k_pages"], s["v_pages"], s["ctx_out"])
    return {k: s[k] for k in _OUTPUTS[op]}


_OUTPUTS = {"tables": ("held_out", "n_free_out", "block_table", "free_list", "start", "slot", "pos"),
            "rope": ("q", "k_pages", "v_pages"), "attend": ("o", "lse"),
            "commit": ("k_pages", "v_pages", "ctx_out")}


# ---- the definitions, in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "attend": _exact_attend,
            "commit": _exact_commit}[case["op"]](case, s)


def _exact_tables(case, s):
    """A server's lists, request after request."""
    page = case["page"]
    table, stack = s["block_table"].cpu().numpy(), s["free_list"].tolist()
    held, n = s["held"].tolist(), int(s["n_free"])
    want = [(t + k + page - 1) // page for t, k in zip(s["ctx"], s["new"])]
    for b, (h, w) in enumerate(zip(held, want)):
        for j in range(w, h):
            stack[n] = int(table[b, j])
            n += 1
    for b, (h, w) in enumerate(zip(held, want)):
        for j in range(h, w):
            n -= 1
            table[b, j] = stack[n]
    start, slot, pos = [0], [], []
    for b, (t, k) in enumerate(zip(s["ctx"], s["new"])):
        for p in range(t, t + k):
            slot.append(int(table[b, p // page]) * page + p % page)
            pos.append(p)
        start.append(len(pos))
    rest = [-1] * (s["M"] - len(pos))
    return {"held_out": _i32(want), "n_free_out": _i32([n]), "block_table": torch.from_numpy(table).cuda(),
            "free_list": _i32(stack), "start": _i32(start), "slot": _i32(slot + rest),
            "pos": _i32(pos + rest)}


def _exact_rope(case, s):
    Hq, Hkv, rot, page = (case[k] for k in ("Hq", "Hkv", "rot", "page"))
    out = {"q": s["q"].double(), "k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
    rows = torch.nonzero(s["slot"] >= 0)[:, 0]
    place = s["slot"][rows].long()
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    first = range(rot // 2) if case["pairing"] == "halves" else range(0, rot, 2)
    second = [i + rot // 2 for i in first] if case["pairing"] == "halves" else [i + 1 for i in first]
    for l in range(case["L"]):
        for h in range(Hq + 2 * Hkv):
            x = s["qkv"][l, rows, h].double()
            if h < Hq + Hkv:
                w = (s["q_weight"] if h < Hq else s["k_weight"])[l].double()
                y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dh"] + 1e-6) * w
                x = y.clone()
                turn = torch.stack([s["pos"][a][rows] for a in axis], -1).double() * s["inv_freq"].double()
                z = torch.polar(torch.ones_like(turn), turn) * torch.complex(y[:, list(first)], y[:, second])
                x[:, list(first)], x[:, second] = z.real, z.imag
            if h < Hq:
                out["q"][l, rows, h] = x
            elif h < Hq + Hkv:
                out["k_pages"][l, place // page, place % page, h - Hq] = x
            else:
                out["v_pages"][l, place // page, place % page, h - Hq - Hkv] = x
    return out


def _up(parent, n):
    """Node n's root-to-node path."""
    path = []
    while n >= 0:
        path.append(n)
        n = parent[n]
    return path[::-1]


def _exact_attend(case, s):
    L, Hq, Hkv, dh, page = (case[k] for k in ("L", "Hq", "Hkv", "dh", "page"))
    G, at = Hq // Hkv, 0
    o, lse = s["o"].double(), s["lse"].double()
    for b, (t, n) in enumerate(zip(s["ctx"], s["new"])):
        places = torch.arange(t + n, device="cuda")
        pg, off = s["block_table"][b].long()[places // page], places % page
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            seen = t + (n if case["tree"] else i1)
            allowed = np.zeros((i1 - i0, seen), dtype=bool)
            for i in range(i0, i1):
                allowed[i - i0, :t] = True
                allowed[i - i0, [t + m for m in _up(s["parents"][b], i)] if case["tree"]
                        else slice(t, t + i + 1)] = True
            hide = torch.from_numpy(~allowed).cuda()
            for l in range(L):
                for h in range(Hkv):
                    q = s["q"][l, at + i0:at + i1, h * G:(h + 1) * G].double()
                    k = s["k_pages"][l, pg[:seen], off[:seen], h].double()
                    v = s["v_pages"][l, pg[:seen], off[:seen], h].double()
                    x = torch.einsum("igd,td->igt", q, k) / math.sqrt(dh)
                    x.masked_fill_(hide[:, None], -math.inf)
                    z = torch.logsumexp(x, -1)
                    lse[l, at + i0:at + i1, h * G:(h + 1) * G] = z
                    o[l, at + i0:at + i1, h * G:(h + 1) * G] = torch.einsum(
                        "igt,td->igd", torch.exp(x - z[..., None]), v)
        at += n
    return {"o": o, "lse": lse}


def _exact_commit(case, s):
    """Node after node of each path, root first."""
    page, ctx_out = case["page"], list(s["ctx"])
    table = s["block_table"].tolist()
    for b, t in enumerate(s["ctx"]):
        path = _up(s["parents"][b], s["ends"][b])
        for i, m in enumerate(path):
            to, frm = (table[b][(t + j) // page] * page + (t + j) % page for j in (i, m))
            for pages in (s["k_pages"], s["v_pages"]):
                pages[:, to // page, to % page] = pages[:, frm // page, frm % page].clone()
        ctx_out[b] = t + len(path)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "ctx_out": _i32(ctx_out)}
