"""Serving with a bounded, shared KV cache: verify rounds of a few chats that
share a system prompt.

Every round, for each of the requests: the draft's top-K scores become a tree
(lbx_ddtree_build), the tree's queries attend to the shared prompt, the
request's own cache and their root paths (lbx_prefix_attention), the target's
choices walk the tree (lbx_accept_walk), the accepted path's attention weights
are added to the cached keys' sums (lbx_attention_mass), and the accepted
nodes' keys and values join the cache, which keeps its budget of entries
(lbx_cache_evict).  For comparison the same queries also run through a sliding
window with a few first positions visible (lbx_window_attention), over a second
cache that holds every position in order: a window counts places, so it cannot
run over a cache that entries have been dropped from.  With a budget that is
never reached lbx_cache_evict only appends.  Queries, keys, logits and draft
scores are synthetic; everything stays on the device.

    python examples/bounded_cache.py [--rounds 20] [--budget 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tree_verify_linear_gb300 import lbx  # noqa: E402

L, BQ, N, HQ, HKV, DH = 4, 5, 22, 24, 4, 256  # layers, requests, nodes, heads, dimension
PROMPT, VOCAB, DEPTH, TOPK = 1024, 1000, 8, 4
WINDOW, SINKS, RECENT = 128, 4, 32


def serve(rounds, budget):
    """The caches, their lengths and the last round's arrays, by name."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    i32 = {"dtype": torch.int32, "device": "cuda"}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    cfg = lbx.make_attn_cfg(L, BQ, N, HQ, HKV, DH, T=budget, P=PROMPT)
    whole = rounds * (DEPTH + 1)  # every token of every round
    win = lbx.make_attn_cfg(L, BQ, N, HQ, HKV, DH, T=whole, window=WINDOW, n_sink=SINKS)
    keep = lbx.make_attn_cfg(L, BQ, N, HQ, HKV, DH, T=budget, n_sink=SINKS)
    ws, win_ws = lbx.new_cache_attn_workspace(cfg), lbx.new_cache_attn_workspace(win)
    walk_ws = lbx.new_accept_workspace(BQ, N, VOCAB)

    k_prompt, v_prompt = normal(L, PROMPT, HKV, DH), normal(L, PROMPT, HKV, DH)
    k_cache, v_cache = normal(L, BQ, budget, HKV, DH), normal(L, BQ, budget, HKV, DH)
    score, pos = torch.zeros(L, BQ, HKV, budget, device="cuda"), torch.zeros(L, BQ, HKV, budget, **i32)
    k_all, v_all = normal(L, BQ, whole, HKV, DH), normal(L, BQ, whole, HKV, DH)
    score_all, pos_all = torch.zeros(L, BQ, HKV, whole, device="cuda"), torch.zeros(L, BQ, HKV, whole, **i32)
    len_all, len_all2 = torch.zeros(BQ, **i32), torch.empty(BQ, **i32)
    ctx, seen = torch.zeros(BQ, **i32), torch.zeros(BQ, **i32)
    ctx2, seen2 = torch.empty(BQ, **i32), torch.empty(BQ, **i32)
    root, status = torch.zeros(BQ, **i32), torch.zeros(1, **i32)
    parent, token, n_nodes = torch.empty(BQ, N, **i32), torch.empty(BQ, N, **i32), torch.empty(BQ, **i32)
    accepted, nxt = torch.empty(BQ, **i32), torch.empty(BQ, **i32)
    o = torch.empty(L, BQ, N, HQ, DH, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(L, BQ, N, HQ, device="cuda")
    score_tree = torch.empty(L, BQ, HKV, N, device="cuda")
    o_win = torch.empty_like(o)

    for r in range(rounds):
        # the draft: top-K tokens per position, and the tree of the best N paths
        p = torch.rand(BQ, DEPTH, TOPK, generator=gen, device="cuda").sort(-1, descending=True).values
        tok = torch.randint(VOCAB, (BQ, DEPTH, TOPK), generator=gen, **i32)
        lbx.lbx_ddtree_build(p.log(), tok, root, N, parent, token, n_nodes)
        # the target's attention over prompt, cache and tree
        q, k_tree, v_tree = normal(L, BQ, N, HQ, DH), normal(L, BQ, N, HKV, DH), normal(L, BQ, N, HKV, DH)
        lbx.lbx_prefix_attention(cfg, ctx, parent, q, k_prompt, v_prompt, k_cache, v_cache, k_tree,
                                 v_tree, o, ws, lse=lse, d_status=status)
        lbx.lbx_window_attention(win, len_all, parent, q, k_all, v_all, k_tree, v_tree, o_win,
                                 win_ws, d_status=status)
        # the target's choices: at most nodes the draft token of a child, so that paths are accepted
        logits = torch.randn(BQ, N, VOCAB, generator=gen, device="cuda")
        parents = torch.where(parent >= 0, parent, N).long()
        nodes = torch.arange(N, device="cuda").expand(BQ, N)
        child = torch.zeros(BQ, N + 1, dtype=torch.long, device="cuda")
        child.scatter_reduce_(1, parents, nodes, "amax")  # the last child; 0 where there is none
        agree = 20.0 * (torch.rand(BQ, N, 1, generator=gen, device="cuda") < 0.8)
        logits.scatter_add_(2, token.long().gather(1, child[:, :N])[..., None], agree)
        lbx.lbx_accept_walk(logits, token, parent, accepted, nxt, walk_ws, d_status=status)
        # upkeep of the cache
        lbx.lbx_attention_mass(cfg, ctx, parent, accepted, q, lse, k_cache, k_tree, score, score_tree,
                               d_status=status)
        lbx.lbx_cache_evict(keep, budget, RECENT, ctx, seen, parent, accepted, k_tree, v_tree,
                            score_tree, k_cache, v_cache, score, pos, ctx2, seen2, d_status=status)
        lbx.lbx_cache_evict(win, whole, 0, len_all, seen, parent, accepted, k_tree, v_tree,
                            score_tree, k_all, v_all, score_all, pos_all, len_all2, seen2,
                            d_status=status)
        last = {"parent": parent, "q": q, "k_tree": k_tree, "v_tree": v_tree, "ctx_len": len_all}
        ctx, ctx2, seen, seen2, root, nxt = ctx2, ctx, seen2, seen, nxt, root
        len_all, len_all2 = len_all2, len_all
    assert int(status.item()) == 0
    return dict(last, seen=seen, ctx=ctx, o=o, o_win=o_win, k_all=k_all, v_all=v_all, pos_all=pos_all,
                len_all=len_all)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--rounds", type=int, default=20)
    ap.add_argument("--budget", type=int, default=256, help="cached entries per request and KV head")
    a = ap.parse_args(argv)
    s = serve(a.rounds, a.budget)
    print(f"{a.rounds} rounds: tokens seen {s['seen'].tolist()}, entries cached {s['ctx'].tolist()}")
    return s["seen"], s["ctx"], s["o"], s["o_win"]


if __name__ == "__main__":
    main()
