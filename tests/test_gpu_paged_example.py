"""The paged cache's example with trees of different sizes: rows are packed, and the last
round's attention is the definition's."""
import os
import sys

import numpy as np
import pytest

import page_ref as R
from test_gpu_paged import built  # noqa: F401

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu

TREES = {"a_budget_that_no_draft_fills": dict(DEPTH=16, TOPK=1), "requests_without_a_draft": dict(MOST=(1, 22, 1)),
         "ragged": dict(MOST=(22, 1, 9)), "small_and_ragged": dict(DEPTH=3, TOPK=1, MOST=(2, 22, 3)),
         "no_drafts": dict(MOST=(1, 1, 1))}


@pytest.mark.parametrize("name", sorted(TREES))
def test_the_example_serves_smaller_trees(name, monkeypatch):
    import paged_cache as P
    for k, v in TREES[name].items():
        monkeypatch.setattr(P, k, v)
    s, out = P.serve(5, 70)
    trie = 1 + sum(P.TOPK ** d for d in range(1, P.DEPTH + 1))
    nodes = [min(P.N, trie, m) for m in P.MOST]
    start = out["start"].tolist()
    assert start == [0] + np.cumsum(nodes).tolist()
    ctx, held = s.ctx.tolist(), s.held.tolist()
    assert int(s.n_free) + sum(held) == P.N_PAGES
    assert all(p + 5 <= c <= p + 5 * min(n, P.DEPTH + 1) for c, p, n in zip(ctx, P.PROMPTS, nodes))
    if max(nodes) > 1:
        assert sum(ctx) > sum(P.PROMPTS) + 15  # some drafts were accepted
    parent = out["parent"].tolist()
    assert all(parent[a] == -1 for a in start[:-1]) and parent[start[-1]:] == [-1] * (len(parent) - start[-1])
    inp = {k: out[k].cpu() for k in ("start", "ctx_len", "block_table", "parent", "q", "k_pages", "v_pages")}
    ref, ref_lse, tol, lse_tol = R.attention(inp)
    live = start[-1]
    assert (np.abs(out["o"].cpu().double().numpy() - ref)[:, :live] <= tol[:, :live]).all()
    assert (np.abs(out["lse"].cpu().double().numpy() - ref_lse)[:, :live] <= lse_tol[:, :live]).all()
