"""The operators of the bounded, shared KV cache in 64 bits, written out from
their definitions one query, key and entry at a time, with the error bounds
the GPU results are held to.

Error bounds.  u is the unit roundoff of the 16-bit type (2^-9 for bf16, 2^-11
for f16).  A score is a sum of dh exact products accumulated in fp32: its error
is at most e = (dh + 2) 2^-24 sum |q||k| scale, taken at the largest sum of the
case, and a weight's relative error at most 2 e + 2^-20 (numerator and
denominator; the exponential is good to 2^-22).  The weights enter the product
with v rounded to the 16-bit type (u each; in f16, weights below the normal
range add 2^-25 of the row's largest), and o is rounded once (u):
    |o - o_ref| <= u |o_ref| + (u + 2 e + 2^-20) sum w |v| + [f16] 2^-25 sum |v|.
lse takes e, the roundings of a log of base 2 and its product (2^-22 of |lse|
each) and of the sum.  Accumulated weights add one fp32 rounding per term.
"""
import numpy as np
import torch

U = {"bf16": 2.0 ** -9, "f16": 2.0 ** -11}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}


def root_path(parent, n):
    path = []
    while n >= 0:
        path.append(int(n))
        n = parent[n]
    return path[::-1]


def visible(parent, n, ctx, window, n_sink):
    """Cached positions and tree nodes that node n's query sees."""
    path = root_path(parent, n)
    at = ctx + len(path) - 1

    def ok(j):
        return window == 0 or at - j < window or j < n_sink
    return [j for j in range(ctx) if ok(j)], [m for d, m in enumerate(path) if ok(ctx + d)]


def attention(inp, window=0, n_sink=0, scale=None, prefix=False):
    """o, lse in fp64 and the bounds of their errors, all [L][Bq][N][Hq](dh)."""
    q = inp["q"].double().numpy()
    kc, vc, kt, vt = (inp[k].double().numpy() for k in ("k_cache", "v_cache", "k_tree", "v_tree"))
    L, Bq, N, Hq, dh = q.shape
    G = Hq // kc.shape[3]
    scale = dh ** -0.5 if scale is None else scale
    f16 = inp["q"].dtype == torch.float16
    u = U["f16" if f16 else "bf16"]
    o, lse = np.zeros_like(q), np.zeros(q.shape[:-1])
    o_tol, lse_tol = np.zeros_like(q), np.zeros(q.shape[:-1])
    for l in range(L):
        for b in range(Bq):
            for n in range(N):
                js, ms = visible(inp["parent"][b].tolist(), n, int(inp["ctx_len"][b]), window, n_sink)
                for h in range(Hq):
                    g = h // G
                    k = np.concatenate([kc[l, b, js, g], kt[l, b, ms, g]])
                    v = np.concatenate([vc[l, b, js, g], vt[l, b, ms, g]])
                    if prefix:
                        k = np.concatenate([inp["k_prefix"][l, :, g].double().numpy(), k])
                        v = np.concatenate([inp["v_prefix"][l, :, g].double().numpy(), v])
                    s = k @ q[l, b, n, h] * scale
                    e = (dh + 2) * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[l, b, n, h])).max()
                    m = s.max()
                    w = np.exp(s - m)
                    total = w.sum()
                    w /= total
                    o[l, b, n, h] = w @ v
                    lse[l, b, n, h] = m + np.log(total)
                    spread = w @ np.abs(v)
                    tol = u * np.abs(o[l, b, n, h]) + (u + 2 * e + 2.0 ** -20) * spread
                    if f16:
                        tol += 2.0 ** -25 * (np.abs(v).sum(0) + 1)
                    o_tol[l, b, n, h] = 1.02 * tol
                    lse_tol[l, b, n, h] = e + 2.0 ** -20 + 2.0 ** -20 * abs(lse[l, b, n, h])
    return o, lse, o_tol, lse_tol


def attention_dense(inp, window=0, n_sink=0):
    """attention() for long caches, as dense masked products in fp64 on the GPU;
    a prefix is taken as the cache's first positions."""
    q = inp["q"].cuda().double()
    L, Bq, N, Hq, dh = q.shape
    Hkv, T = inp["k_tree"].shape[3], inp["k_cache"].shape[2]
    G, u = Hq // Hkv, U["f16" if inp["q"].dtype == torch.float16 else "bf16"]
    P = inp["k_prefix"].shape[1] if "k_prefix" in inp else 0
    seen = torch.zeros(Bq, N, P + T + N, dtype=torch.bool)
    seen[:, :, :P] = True
    for b in range(Bq):
        for n in range(N):
            js, ms = visible(inp["parent"][b].tolist(), n, int(inp["ctx_len"][b]), window, n_sink)
            seen[b, n, [P + j for j in js] + [P + T + m for m in ms]] = True
    seen = seen.cuda().repeat_interleave(G, 1)
    o, lse = torch.empty_like(q), torch.empty(L, Bq, N, Hq, dtype=torch.float64, device="cuda")
    o_tol, lse_tol = torch.empty_like(q), torch.empty_like(lse)
    for l in range(L):
        for g in range(Hkv):
            parts = [[inp[c][l, :, :, g] for c in (x + "_cache", x + "_tree")] for x in "kv"]
            if P:
                parts = [[inp[x + "_prefix"][l, None, :, g].expand(Bq, -1, -1)] + p
                         for x, p in zip("kv", parts)]
            k, v = (torch.cat(p, 1).cuda().double() for p in parts)
            qg = q[l, :, :, g * G:(g + 1) * G].reshape(Bq, N * G, dh)
            s = (qg @ k.transpose(1, 2) * dh ** -0.5).masked_fill(~seen, -torch.inf)
            e = (qg.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(-1)
            e = e * (dh ** -0.5 * (dh + 2) * 2.0 ** -24)
            z = s.logsumexp(-1)
            w = (s - z[..., None]).exp()
            o1 = w @ v
            t1 = 1.02 * (u * o1.abs() + (u + 2 * e[..., None] + 2.0 ** -20) * (w @ v.abs()))
            if inp["q"].dtype == torch.float16:
                t1 += 1.02 * 2.0 ** -25 * (seen.double() @ v.abs() + 1)
            o[l, :, :, g * G:(g + 1) * G] = o1.view(Bq, N, G, dh)
            o_tol[l, :, :, g * G:(g + 1) * G] = t1.view(Bq, N, G, dh)
            lse[l, :, :, g * G:(g + 1) * G] = z.view(Bq, N, G)
            lse_tol[l, :, :, g * G:(g + 1) * G] = (e + 2.0 ** -20 * (1 + z.abs())).view(Bq, N, G)
    return o.cpu().numpy(), lse.cpu().numpy(), o_tol.cpu().numpy(), lse_tol.cpu().numpy()


def mass(inp, lse, score, window=0, n_sink=0, scale=None):
    """score, score_tree in fp64 and the bounds of their errors."""
    q, kc, kt = (inp[k].double().numpy() for k in ("q", "k_cache", "k_tree"))
    L, Bq, N, Hq, dh = q.shape
    Hkv = kc.shape[3]
    G = Hq // Hkv
    scale = dh ** -0.5 if scale is None else scale
    out = score.astype(np.float64).copy()
    tree = np.zeros((L, Bq, Hkv, N))
    tol, tree_tol = 2.0 ** -22 * np.abs(out), np.zeros_like(tree)
    for l in range(L):
        for b in range(Bq):
            parent, ctx = inp["parent"][b].tolist(), int(inp["ctx_len"][b])
            for n in root_path(parent, int(inp["accepted"][b])):
                js, ms = visible(parent, n, ctx, window, n_sink)
                for h in range(Hq):
                    z = float(lse[l, b, n, h])
                    if z == -np.inf:
                        continue
                    for keys, idx, dst, dtol in ((kc, js, out, tol), (kt, ms, tree, tree_tol)):
                        k = keys[l, b, idx, h // G]
                        if not len(idx):
                            continue
                        e = (dh + 2) * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[l, b, n, h])).max()
                        w = np.exp(k @ q[l, b, n, h] * scale - z)
                        dst[l, b, h // G, idx] += w
                        # one more rounding for each term summed before or after
                        dtol[l, b, h // G, idx] += w * (e + (abs(z) + 4) * 2.0 ** -21 + N * G * 2.0 ** -24)
    return out, tree, tol + 1e-30, tree_tol + 1e-30


def mass_dense(inp, lse, score):
    """mass() for long caches without a window, as dense products in fp64 on the GPU."""
    q = inp["q"].cuda().double()
    L, Bq, N, Hq, dh = q.shape
    Hkv, T = inp["k_tree"].shape[3], inp["k_cache"].shape[2]
    G = Hq // Hkv
    out, tree = score.astype(np.float64), np.zeros((L, Bq, Hkv, N))
    tol, tree_tol = 2.0 ** -22 * np.abs(out) + 1e-30, np.full(tree.shape, 1e-30)
    for b in range(Bq):
        ctx = int(inp["ctx_len"][b])
        path = root_path(inp["parent"][b].tolist(), int(inp["accepted"][b]))
        seen = torch.ones(len(path), G, ctx + len(path), dtype=torch.bool)
        seen[:, :, ctx:] = torch.ones(len(path), len(path), dtype=torch.bool).tril()[:, None]
        for l in range(L):
            for g in range(Hkv):
                k = torch.cat([inp["k_cache"][l, b, :ctx, g], inp["k_tree"][l, b, path, g]]).cuda().double()
                qp = q[l, b, path, g * G:(g + 1) * G]
                z = torch.from_numpy(lse[l, b, path, g * G:(g + 1) * G]).cuda().double()[..., None]
                w = (qp @ k.T * dh ** -0.5 - z).exp().masked_fill(~seen.cuda(), 0)
                e = (qp.abs() @ k.abs().T).amax(-1, keepdim=True) * (dh ** -0.5 * (dh + 2) * 2.0 ** -24)
                t = (w * (e + (z.abs() + 4) * 2.0 ** -21 + N * G * 2.0 ** -24)).sum((0, 1)).cpu().numpy()
                w = w.sum((0, 1)).cpu().numpy()
                out[l, b, g, :ctx] += w[:ctx]
                tol[l, b, g, :ctx] += t[:ctx]
                tree[l, b, g, path], tree_tol[l, b, g, path] = w[ctx:], t[ctx:] + 1e-30
    return out, tree, tol, tree_tol


def evict(inp, score, score_tree, pos, seen, budget, n_sink, n_recent):
    """New copies of k_cache, v_cache, score, pos, and ctx_out, seen_out."""
    kc, vc = inp["k_cache"].clone(), inp["v_cache"].clone()
    score, pos = score.copy(), pos.copy()
    L, Bq, T, Hkv, _ = kc.shape
    ctx_out, seen_out = [], []
    for b in range(Bq):
        ctx = int(inp["ctx_len"][b])
        path = root_path(inp["parent"][b].tolist(), int(inp["accepted"][b]))
        n, end = ctx + len(path), int(seen[b]) + len(path)
        size = min(n, budget)
        ctx_out.append(size)
        seen_out.append(end)
        for l in range(L):
            for g in range(Hkv):
                p = list(pos[l, b, g, :ctx]) + [int(seen[b]) + d for d in range(len(path))]
                s = list(score[l, b, g, :ctx]) + [score_tree[l, b, g, m] for m in path]

                def rank(i):
                    if p[i] < n_sink or p[i] >= end - n_recent:
                        return (0, 0.0, i)
                    return (2, 0.0, i) if np.isnan(s[i]) else (1, -float(s[i]), i)
                keep = sorted(sorted(range(n), key=rank)[:size])
                stay = {i for i in keep if i < min(ctx, size)}
                free = [z for z in range(size) if z not in stay]
                for i, z in zip([i for i in keep if i not in stay], free):
                    old = i < ctx
                    kc[l, b, z, g] = inp["k_cache"][l, b, i, g] if old else inp["k_tree"][l, b, path[i - ctx], g]
                    vc[l, b, z, g] = inp["v_cache"][l, b, i, g] if old else inp["v_tree"][l, b, path[i - ctx], g]
                    score[l, b, g, z], pos[l, b, g, z] = s[i], p[i]
    return kc, vc, score, pos, np.array(ctx_out, np.int32), np.array(seen_out, np.int32)


def make_inputs(L, Bq, N, Hq, Hkv, dh, T, P=0, dtype="bf16", ctx=None, tree="random", seed=0,
                width=2.0):
    """Seeded inputs on the CPU: q wider than the keys, so that weights gather."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g).to(DTYPE[dtype])
    if ctx is None:
        ctx = [int(rng.integers(0, T + 1)) for _ in range(Bq)]
    parent = np.full((Bq, N), -1, np.int32)
    for b in range(Bq):
        for i in range(1, N):
            parent[b, i] = i - 1 if tree == "chain" else 0 if tree == "star" else rng.integers(0, i)
    inp = {"q": (normal(L, Bq, N, Hq, dh) * width), "k_cache": normal(L, Bq, T, Hkv, dh),
           "v_cache": normal(L, Bq, T, Hkv, dh), "k_tree": normal(L, Bq, N, Hkv, dh),
           "v_tree": normal(L, Bq, N, Hkv, dh), "ctx_len": torch.tensor(ctx, dtype=torch.int32),
           "parent": torch.from_numpy(parent),
           "accepted": torch.from_numpy(rng.integers(0, N, Bq).astype(np.int32))}
    if P:
        inp["k_prefix"], inp["v_prefix"] = normal(L, P, Hkv, dh), normal(L, P, Hkv, dh)
    return inp
