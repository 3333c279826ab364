"""The operators of the paged KV cache in 64 bits, written out from their
definitions one request, row and key at a time, with the error bounds the GPU
results are held to.

Error bounds.  u is half a step of the 16-bit type relative to the value (2^-8 for
bf16, 2^-11 for f16).

Rotation.  In units of 2^-24 relative to the values: the mean of squares and its
root 8 (dh additions in fp32 in shuffled pairs: log2(dh) of them deep, halved by
the root; eps, root and quotient), two products with the weight 2, cosine and sine
4 and the angle's fraction of a turn 2^-24 pi at most, two products and a sum 3.
All of it stays below 32 2^-24 (|a| + |b|) of the pair; then the result is rounded
once: |y - y_ref| <= u |y_ref| + 1.01 * 2^-19 (|a| + |b|).  Values are copies.

Attention.  As for the bounded cache (cache_ref): a score's error is at most
e = (dh + 2) 2^-24 sum |q||k| scale, a weight's relative error 2 e + 2^-20; the weights
meet v rounded to the 16-bit type (u each; f16 weights below the normal range add
2^-25 of the row's largest) and o is rounded once:
    |o - o_ref| <= u |o_ref| + (u + 2 e + 2^-20) sum w |v| + [f16] 2^-25 sum |v|.
lse takes e, and 2^-20 of 1 + |lse|.  A long sum in fp32 adds 2^-24 per term that
follows; at most T terms: sums of more than 2^12 keys get T 2^-24 besides.
"""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}


def root_path(parent, n):
    path = []
    while n >= 0:
        path.append(int(n))
        n = int(parent[n])
    return path[::-1]


def tree(rng, n, kind="random"):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    return [-1] + [int(rng.integers(0, i)) for i in range(1, n)]


def pages_of(t, page):
    return -(-t // page)


def make_batch(ctx, new, page, seed=0, spare=2, wide=1):
    """Pages of requests with ctx cached and new tokens each, in a random order;
    table columns past a request's pages name pages that do not exist."""
    rng = np.random.default_rng(seed)
    need = [pages_of(t + n, page) for t, n in zip(ctx, new)]
    n_pages = sum(need) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(ctx), max(need + [0]) + wide), -7, dtype=np.int32)
    at = 0
    for b, h in enumerate(need):
        table[b, :h] = order[at:at + h]
        at += h
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return rng, n_pages, table, start


def place(table, b, p, page):
    return int(table[b, p // page]), p % page


def make_attention(ctx, new, Hq, Hkv, dh, page, L=1, dtype="bf16", kind=None, pad=0, seed=0, width=2.0):
    """Inputs on the CPU; whatever no query sees is NaN."""
    rng, n_pages, table, start = make_batch(ctx, new, page, seed)
    g = torch.Generator().manual_seed(seed)
    dt = DTYPE[dtype]
    M = int(start[-1]) + pad
    shape = (L, n_pages, page, Hkv, dh)
    k, v = torch.full(shape, float("nan"), dtype=dt), torch.full(shape, float("nan"), dtype=dt)
    for b, (t, n) in enumerate(zip(ctx, new)):
        for j in range(pages_of(t + n, page)):
            rows = min(page, t + n - j * page)
            for pool in (k, v):
                pool[:, table[b, j], :rows] = torch.randn(L, rows, Hkv, dh, generator=g).to(dt)
    q = (torch.randn(L, M, Hq, dh, generator=g) * width).to(dt)
    parent = None
    if kind:
        parent = [p for n in new if n for p in tree(rng, n, kind)] + [-5] * pad
        parent = torch.tensor(parent, dtype=torch.int32)
    return {"start": torch.from_numpy(start), "ctx_len": torch.tensor(ctx, dtype=torch.int32),
            "block_table": torch.from_numpy(table), "parent": parent, "q": q, "k_pages": k, "v_pages": v}


def attention(inp, scale=None, device="cpu"):
    """o, lse in fp64 and the bounds of their errors; rows of padding are NaN."""
    q = inp["q"].to(device).double()
    L, M, Hq, dh = q.shape
    page, Hkv = inp["k_pages"].shape[2:4]
    G, u, f16 = Hq // Hkv, U[inp["q"].dtype], inp["q"].dtype == torch.float16
    scale = dh ** -0.5 if scale is None else scale
    start, ctx = inp["start"].tolist(), inp["ctx_len"].tolist()
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan")).to(q)
    o_tol, lse_tol = o.clone(), lse.clone()
    for b, t in enumerate(ctx):
        s, n = start[b], start[b + 1] - start[b]
        if n == 0:
            continue
        table = inp["block_table"][b].long()
        p = torch.arange(t + n)
        pg, off = table[p // page], p % page
        k_all = inp["k_pages"][:, pg, off].to(device).double()
        v_all = inp["v_pages"][:, pg, off].to(device).double()
        seen = torch.zeros(n, t + n, dtype=torch.bool)
        for i in range(n):
            seen[i, :t] = True
            own = (range(i + 1) if inp["parent"] is None
                   else root_path(inp["parent"][s:s + n].tolist(), i))
            seen[i, [t + m for m in own]] = True
        seen = seen.to(device)[:, None]
        for l in range(L):
            for g in range(Hkv):
                k, v = k_all[l, :, g], v_all[l, :, g]
                qg = q[l, s:s + n, g * G:(g + 1) * G]
                x = (qg @ k.t() * scale).masked_fill(~seen, -torch.inf)
                e = ((qg.abs() @ k.abs().t()).masked_fill(~seen, 0).amax(-1, keepdim=True)
                     * scale * (dh + 2) * 2.0 ** -24)
                z = x.logsumexp(-1, keepdim=True)
                w = (x - z).exp()
                far = (t + n) * 2.0 ** -24 if t + n > 4096 else 0.0
                ref = w @ v
                tol = u * ref.abs() + (u + 2 * e + 2.0 ** -20 + far) * (w @ v.abs())
                if f16:
                    tol += 2.0 ** -25 * (seen.double() @ v.abs() + 1)
                at = (l, slice(s, s + n), slice(g * G, (g + 1) * G))
                o[at], o_tol[at] = ref, 1.02 * tol
                lse[at], lse_tol[at] = z[..., 0], (e + 2.0 ** -20 * (1 + z.abs()) + far)[..., 0]
    return tuple(x.cpu().numpy() for x in (o, lse, o_tol, lse_tol))


def rope(x, weight, inv_freq, pos, sections, pairing, eps):
    """Head rows x [M][H][dh] (any float type) turned, in fp64, and the bound of the
    error before the last rounding."""
    y = x.double().numpy().copy()
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * weight.double().numpy()
    out, tol = y.copy(), np.abs(y) * 1.01 * 2.0 ** -19
    half = sum(sections)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for i in range(half):
        a, b = (i, i + half) if pairing == "halves" else (2 * i, 2 * i + 1)
        t = pos[axis[i]].double().numpy() * float(inv_freq[i])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        tol[..., a] = tol[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * 1.01 * 2.0 ** -19
    return out, tol


def tables(ctx, new, held, n_free, table, stack, page, M):
    """A server's lists, request after request."""
    table, stack, top = table.copy(), stack.copy(), n_free
    want = [pages_of(t + n, page) for t, n in zip(ctx, new)]
    for b, (h, w) in enumerate(zip(held, want)):
        for j in range(w, h):
            stack[top] = table[b, j]
            top += 1
    for b, (h, w) in enumerate(zip(held, want)):
        for j in range(h, w):
            top -= 1
            table[b, j] = stack[top]
    start, slot, pos = [0], [-1] * M, [-1] * M
    for b, (t, n) in enumerate(zip(ctx, new)):
        for i in range(n):
            r = start[-1] + i
            slot[r], pos[r] = int(table[b, (t + i) // page]) * page + (t + i) % page, t + i
        start.append(start[-1] + n)
    return {"held_out": want, "n_free_out": [top], "block_table": table, "free_list": stack,
            "start": start, "slot": slot, "pos": pos}
