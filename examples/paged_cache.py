"""Serving with a paged KV cache: prompts in chunks, then verify rounds of draft trees.

The requests' keys and values lie in pages of one pool.  Every step gives the
requests the pages that their lengths need and takes back the others
(lbx_page_tables), norms and turns the new tokens' queries and keys and puts keys
and values into their pages (lbx_qk_norm_rope), and attends over the pages
(lbx_paged_attention).  Prompts come in chunks of tokens; after them every
request verifies a draft tree per round: the draft's top-K scores become a tree
(lbx_ddtree_build), the target's choices walk it (lbx_accept_walk), and the
accepted path stays in the cache (lbx_page_commit).  The tree's arrays have N nodes per
request, unused ones at the end; the paged calls take rows without gaps, so that nodes are
packed on the way (a draft of few candidates gives a smaller tree, and a request may
have a smaller budget, 1 for none).  Projections, logits and draft
scores are synthetic; everything stays on the device.

    python examples/paged_cache.py [--rounds 10] [--chunk 96]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tree_verify_linear_gb300 import lbx  # noqa: E402

L, BQ, N, HQ, HKV, DH = 2, 3, 22, 24, 4, 256  # layers, requests, nodes, heads, dimension
PAGE, N_PAGES, WIDTH, ROT = 64, 48, 16, 64
VOCAB, DEPTH, TOPK = 1000, 8, 4
PROMPTS = (300, 77, 150)
MOST = (N, N, N)  # nodes that each request's tree may have


class Server:
    def __init__(self, seed=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        i32 = self.i32 = {"dtype": torch.int32, "device": "cuda"}
        self.table = torch.zeros(BQ, WIDTH, **i32)
        self.stack = torch.arange(N_PAGES, **i32)
        self.held, self.n_free = torch.zeros(BQ, **i32), torch.full((1,), N_PAGES, **i32)
        self.held2, self.n_free2 = torch.zeros(BQ, **i32), torch.zeros(1, **i32)
        shape = (L, N_PAGES, PAGE, HKV, DH)
        self.k_pages, self.v_pages = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.ctx, self.ctx2 = torch.zeros(BQ, **i32), torch.zeros(BQ, **i32)
        self.status = torch.zeros(1, **i32)
        self.inv_freq = (1e7 ** (-torch.arange(ROT // 2, device="cuda").double() / (ROT // 2))).float()
        self.weights = [torch.rand(L, DH, generator=self.gen, device="cuda") + 0.5 for _ in "qk"]
        self.rope = lbx.make_rope_cfg([ROT // 2])
        self.ws = lbx.new_paged_workspace(self.cfg(1))

    def cfg(self, rows):
        return lbx.make_page_cfg(L, BQ, rows, HQ, HKV, DH, PAGE, N_PAGES, WIDTH)

    def step(self, new, rows, parent=None, depth=None):
        """One step of `new` tokens per request (rows of them, padding included): the
        arrays of the step by name."""
        cfg = self.cfg(rows)
        start = torch.zeros(BQ + 1, **self.i32)
        slot, pos = torch.zeros(rows, **self.i32), torch.zeros(1, rows, **self.i32)
        lbx.lbx_page_tables(cfg, self.ctx, new, self.held, self.n_free, self.table, self.stack, self.held2,
                            self.n_free2, start, slot, pos[0], d_status=self.status)
        self.held, self.held2, self.n_free, self.n_free2 = self.held2, self.held, self.n_free2, self.n_free
        if depth is not None:  # a tree's nodes stand at their depth behind the context
            pos = self.pack(self.ctx[:, None] + depth, new).view(1, rows)
            parent = self.pack(parent, new)
        qkv = torch.randn(L, rows, HQ + 2 * HKV, DH, generator=self.gen, device="cuda", dtype=torch.bfloat16)
        q = torch.zeros(L, rows, HQ, DH, dtype=torch.bfloat16, device="cuda")
        lbx.lbx_qk_norm_rope(cfg, self.rope, qkv, self.inv_freq, pos, slot, q, self.k_pages, self.v_pages,
                             q_weight=self.weights[0], k_weight=self.weights[1], d_status=self.status)
        o, lse = torch.zeros_like(q), torch.zeros(L, rows, HQ, device="cuda")
        lbx.lbx_paged_attention(cfg, start, self.ctx, self.table, q, self.k_pages, self.v_pages, o, self.ws,
                                parent=parent, lse=lse, d_status=self.status)
        return {"cfg": cfg, "start": start, "q": q, "o": o, "lse": lse, "parent": parent}

    def pack(self, x, n_nodes):
        """Nodes [BQ][N] as rows: request after request, without the unused ones (-1 behind)."""
        node, end = torch.arange(N, device="cuda"), n_nodes.cumsum(0)
        row = torch.where(node < n_nodes[:, None], (end - n_nodes)[:, None] + node, BQ * N)
        return torch.full((BQ * N + 1,), -1, **self.i32).scatter_(0, row.flatten(), x.flatten())[:-1]

    def prompts(self, chunk):
        left = torch.tensor(PROMPTS, **self.i32)
        while int(left.max()) > 0:
            new = left.clamp(max=chunk)
            self.step(new, BQ * chunk)
            self.ctx = self.ctx + new
            left = left - new

    def round(self, root):
        p = torch.rand(BQ, DEPTH, TOPK, generator=self.gen, device="cuda").sort(-1, descending=True).values
        tok = torch.randint(VOCAB, (BQ, DEPTH, TOPK), generator=self.gen, **self.i32)
        parent, token, depth = (torch.empty(BQ, N, **self.i32) for _ in range(3))
        n_nodes = torch.empty(BQ, **self.i32)
        lbx.lbx_ddtree_build(p.log(), tok, root, N, parent, token, n_nodes, depth_out=depth)
        # the first nodes of a tree are one; the walk takes N nodes: unused ones hang on the root
        # with a token that never matches
        n_nodes = torch.minimum(n_nodes, torch.tensor(MOST, **self.i32))
        nodes = torch.arange(N, device="cuda").expand(BQ, N)
        used = nodes < n_nodes[:, None]
        parent, token = torch.where(used, parent, 0), torch.where(used, token, -1)
        out = self.step(n_nodes, BQ * N, parent=parent, depth=depth)
        # the target's choices: at most nodes the draft token of a child, so that paths are accepted
        logits = torch.randn(BQ, N, VOCAB, generator=self.gen, device="cuda")
        child = torch.zeros(BQ, N + 1, dtype=torch.long, device="cuda")
        child.scatter_reduce_(1, torch.where(used & (parent >= 0), parent, N).long(), nodes, "amax")
        agree = 20.0 * (torch.rand(BQ, N, 1, generator=self.gen, device="cuda") < 0.8)
        logits.scatter_add_(2, token.long().gather(1, child[:, :N])[..., None], agree)
        accepted, nxt = torch.empty(BQ, **self.i32), torch.empty(BQ, **self.i32)
        lbx.lbx_accept_walk(logits, token, parent, accepted, nxt, lbx.new_accept_workspace(BQ, N, VOCAB),
                            d_status=self.status)
        out.update(ctx_len=self.ctx.clone(), k_pages=self.k_pages.clone(), v_pages=self.v_pages.clone(),
                   block_table=self.table.clone(), accepted=accepted)
        lbx.lbx_page_commit(out["cfg"], out["start"], self.ctx, self.table, out["parent"], accepted,
                            self.k_pages, self.v_pages, self.ctx2, d_status=self.status)
        self.ctx, self.ctx2 = self.ctx2, self.ctx
        return nxt, out


def serve(rounds, chunk):
    s = Server()
    s.prompts(chunk)
    root, out = torch.zeros(BQ, **s.i32), None
    for _ in range(rounds):
        root, out = s.round(root)
    assert int(s.status.item()) == 0
    return s, out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--rounds", type=int, default=10)
    ap.add_argument("--chunk", type=int, default=96, help="tokens of a prompt per step and request")
    a = ap.parse_args(argv)
    s, out = serve(a.rounds, a.chunk)
    print(f"{a.rounds} rounds after prompts of {PROMPTS}: {s.ctx.tolist()} tokens in {s.held.tolist()} pages, "
          f"{int(s.n_free)} of {N_PAGES} free")
    return s, out


if __name__ == "__main__":
    main()
