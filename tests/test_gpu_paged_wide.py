"""GPU parity of lbx_paged_attention on pairs of CTAs with two subtiles each, which head
dimension 128 takes when requests bring many rows; bounds as in page_ref."""
import os
import re

import numpy as np
import pytest
import torch

import page_ref as R
from test_gpu_paged import built, check_attention, i32, page_cfg, run_attention, status_word  # noqa: F401
from tree_verify_linear_gb300 import build, lbx

pytestmark = pytest.mark.gpu


def wide(inp):
    """The input, if the host's rule takes pairs for it."""
    with open(os.path.join(build.CSRC, "page_attn.cu")) as f:
        most = int(re.search(r"kWideRows = (\d+);", f.read()).group(1))
    L, M, Hq, dh = inp["q"].shape
    assert dh == 128 and M * (Hq // inp["k_pages"].shape[3]) > most * len(inp["ctx_len"])
    return inp


WIDE = {
    "chunks": dict(ctx=[129, 513], new=[400, 600], Hq=8, Hkv=2, page=128),
    "whole_prompts": dict(ctx=[0, 0], new=[512, 640], Hq=8, Hkv=2, page=64, pad=5),
    "tails": dict(ctx=[5, 0, 300, 64], new=[193, 227, 129, 225], Hq=8, Hkv=2, page=16),
    "beside_single_tokens": dict(ctx=[0, 3000, 77, 9], new=[900, 1, 0, 33], Hq=8, Hkv=2, page=32, pad=7),
    "pieces": dict(ctx=[9000], new=[300], Hq=4, Hkv=1, page=16),
    "layers": dict(ctx=[40, 0], new=[210, 230], Hq=8, Hkv=2, page=16, L=3),
    "group_of_1": dict(ctx=[100], new=[900], Hq=2, Hkv=2, page=256),
    "group_of_7": dict(ctx=[50, 333], new=[200, 130], Hq=14, Hkv=2, page=16),
    "group_of_48": dict(ctx=[70, 3], new=[20, 18], Hq=48, Hkv=1, page=32),
    "group_of_100": dict(ctx=[70, 3], new=[9, 8], Hq=100, Hkv=1, page=32),
    "group_of_128": dict(ctx=[70, 3], new=[7, 9], Hq=128, Hkv=1, page=16),
    "trees": dict(ctx=[300, 0], new=[64, 64], Hq=32, Hkv=2, page=16, kind="random"),
    "trees_group_of_13": dict(ctx=[130], new=[64], Hq=26, Hkv=2, page=32, kind="random", L=2),
    "tree_star": dict(ctx=[63], new=[50], Hq=16, Hkv=1, page=64, kind="star"),
    "trees_over_long_keys": dict(ctx=[5000, 2500], new=[64, 40], Hq=32, Hkv=2, page=64, kind="random"),
    "wide_scores": dict(ctx=[400, 300], new=[300, 270], Hq=8, Hkv=2, page=64, width=20.0),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(WIDE))
def test_pairs(name, dtype):
    check_attention(wide(R.make_attention(**WIDE[name], dh=128, dtype=dtype, seed=400 + len(name))),
                    device="cuda", calls=2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pairs_with_scores_of_minus_infinity_and_nan(dtype):
    inp = wide(R.make_attention([20, 200, 30], [3, 600, 200], 8, 2, 128, 16, dtype=dtype, seed=6))
    clean, clean_lse, _ = run_attention(inp)
    q, k = inp["q"], inp["k_pages"]
    q[:, 0:3] = q[:, 0:3].abs() + 0.5  # request 0: every score -inf
    for p in range(23):
        k[:, inp["block_table"][0, p // 16], p % 16] = -torch.inf
    q[0, 3 + 370, 1, 5] = torch.nan  # request 1, token 370: one head's scores are NaN
    o, lse, status = run_attention(inp)
    assert status == 0
    assert (o[:, :3] == 0).all() and (lse[:, :3] == -torch.inf).all()
    assert o[0, 373, 1].isnan().all() and lse[0, 373, 1].isnan()
    same = torch.ones(o.shape[:3], dtype=torch.bool)
    same[:, :3] = same[0, 373, 1] = False
    assert torch.equal(o[same], clean[same]) and torch.equal(lse[same], clean_lse[same])


@pytest.mark.parametrize("dh,new", [(64, 20), (64, 500), (128, 20), (128, 500), (256, 20), (256, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_keys_of_minus_infinity_among_others(dh, new, dtype):
    """Pages of keys whose scores are all -inf, a first block of nothing else included: o and
    lse are those of a request without them."""
    inp = R.make_attention([320], [new], 8, 2, dh, 16, dtype=dtype, seed=7)
    if (dh, new) == (128, 500):
        wide(inp)
    inp["q"] = inp["q"].abs() + 0.5
    dead = list(range(9)) + [13, 19]
    table = inp["block_table"]
    inp["k_pages"][:, table[0, dead].long()] = -torch.inf
    o, lse, status = run_attention(inp)
    assert status == 0
    alive = [j for j in range(R.pages_of(320 + new, 16)) if j not in dead]
    ref, ref_lse, tol, lse_tol = R.attention(
        dict(inp, block_table=table[:, alive], ctx_len=inp["ctx_len"] - 16 * len(dead)), device="cuda")
    assert (np.abs(o.double().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().numpy() - ref_lse) <= lse_tol).all()


@pytest.mark.parametrize("page_id", [-1, 10 ** 6, 2 ** 31 - 1])
def test_pairs_do_not_read_a_page_outside_the_pool(page_id):
    inp = wide(R.make_attention([40, 7, 500], [9, 800, 1], 8, 2, 128, 16, seed=9))
    clean, clean_lse, _ = run_attention(inp)
    inp["block_table"][1, 3] = page_id
    o, lse, status = run_attention(inp)
    assert status == lbx.LBX_EINVAL
    rest = list(range(9)) + [809]
    assert torch.equal(o[:, rest], clean[:, rest]) and torch.equal(lse[:, rest], clean_lse[:, rest])


BAD = {
    "start_falls": lambda i: i["start"].__setitem__(1, 129),
    "past_the_table": lambda i: i["ctx_len"].__setitem__(1, 16 * i["block_table"].shape[1] - 63),
    "parent_not_before": lambda i: i["parent"].__setitem__(70, 6),
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_pairs_refuse_bad_batches(name):
    inp = wide(R.make_attention([40, 7], [64, 64], 32, 2, 128, 16, kind="random", seed=9))
    BAD[name](inp)
    o, lse, status = run_attention(inp)
    assert status == lbx.LBX_ETREE and (o == 55.0).all() and (lse == 55.0).all()


def test_pairs_in_a_graph_whatever_tokens_come():
    """Captured for many rows, replayed with prompts, chunks, single tokens and nothing."""
    B, M, Hq, Hkv, page, width = 3, 1200, 8, 2, 16, 90
    n_pages = B * width
    g = torch.Generator().manual_seed(1)
    a = {"q": torch.randn(1, M, Hq, 128, generator=g), "k_pages": torch.randn(1, n_pages, page, Hkv, 128, generator=g),
         "v_pages": torch.randn(1, n_pages, page, Hkv, 128, generator=g)}
    a = {k: v.to(torch.bfloat16) for k, v in a.items()}
    a["block_table"] = torch.randperm(n_pages, generator=g).to(torch.int32).view(B, width)
    a["start"], a["ctx_len"] = torch.zeros(B + 1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    a["parent"] = None
    wide(a)
    d = {k: None if v is None else v.cuda() for k, v in a.items()}
    cfg, o, lse = page_cfg(a), torch.zeros_like(d["q"]), torch.zeros(1, M, Hq, device="cuda")
    ws, status = lbx.new_paged_workspace(cfg), status_word()

    def call():
        lbx.lbx_paged_attention(cfg, d["start"], d["ctx_len"], d["block_table"], d["q"], d["k_pages"], d["v_pages"],
                                o, ws, lse=lse, d_status=status)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for ctx, new in (([0, 0, 0], [700, 33, 467]), ([1000, 700, 3], [1, 1, 1]), ([900, 0, 50], [300, 0, 257]),
                     ([5, 5, 5], [0, 0, 0]), ([1300, 1400, 17], [64, 2, 900])):
        a["ctx_len"], a["start"] = torch.tensor(ctx, dtype=torch.int32), torch.tensor(
            [0] + np.cumsum(new).tolist(), dtype=torch.int32)
        d["ctx_len"].copy_(a["ctx_len"]), d["start"].copy_(a["start"])
        o.fill_(55.0), lse.fill_(55.0)
        graph.replay()
        torch.cuda.synchronize()
        ref, ref_lse, tol, lse_tol = R.attention(a, device="cuda")
        live = sum(new)
        assert (np.abs(o.cpu().double().numpy() - ref)[:, :live] <= tol[:, :live]).all()
        assert (np.abs(lse.cpu().double().numpy() - ref_lse)[:, :live] <= lse_tol[:, :live]).all()
        assert (o[:, live:] == 55.0).all() and (lse[:, live:] == 55.0).all()
    assert int(status.item()) == 0
