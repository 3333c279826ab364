"""The paged cache's operators in a pool whose offsets pass 32 bits, and weights in two parts
beside infinities, NaN and pages that do not exist; bounds as in page_ref."""
import numpy as np
import pytest
import torch

import page_ref as R
from test_gpu_paged import (TYPE, built, i32, page_cfg, rope_inputs, run_attention, run_commit, run_rope,  # noqa: F401
                            same_bits, status_word)
from tree_verify_linear_gb300 import lbx

pytestmark = pytest.mark.gpu


def far_pools(inp, n_pages):
    """The input on the device, its pages spread to the far end of pools of n_pages: (arrays,
    where each old page went)."""
    L, old, page, Hkv, dh = inp["k_pages"].shape
    to = torch.tensor([n_pages - 1 - 7 * j for j in range(old)])
    assert L * n_pages * page * Hkv * dh > 2 ** 32 and int(to.min()) > 0
    d = {k: v.cuda() for k, v in inp.items() if isinstance(v, torch.Tensor) and not k.endswith("_pages")}
    for k in ("k_pages", "v_pages"):
        d[k] = torch.empty(L, n_pages, page, Hkv, dh, dtype=inp[k].dtype, device="cuda")
        d[k][:, to.cuda()] = inp[k].cuda()
    return d, to


@pytest.mark.parametrize("dh,page,n_pages", [(256, 64, 2 ** 17), (128, 16, 2 ** 20), (64, 256, 2 ** 17)])
@pytest.mark.parametrize("kind", ["few", "tokens", "chunk", "tree"])
def test_attention_in_a_far_pool(dh, page, n_pages, kind):
    ctx, new = {"few": ([300, 20], [1, 1]), "tokens": ([9000, 5000, 70], [1, 1, 1]),
                "chunk": ([300, 5], [300, 200]), "tree": ([500, 70], [22, 40])}[kind]
    inp = R.make_attention(ctx, new, 8, 2, dh, page, L=2, kind="random" if kind == "tree" else None, seed=11)
    d, to = far_pools(inp, n_pages)
    table = inp["block_table"].long()
    d["block_table"] = torch.where(table >= 0, to[table.clamp(min=0)], -1).to(torch.int32).cuda()
    cfg = lbx.make_page_cfg(2, len(ctx), d["q"].shape[1], 8, 2, dh, page, n_pages, table.shape[1])
    o, lse = torch.zeros_like(d["q"]), torch.zeros(d["q"].shape[:3], device="cuda")
    ws, status = lbx.new_paged_workspace(cfg), status_word()
    lbx.lbx_paged_attention(cfg, d["start"], d["ctx_len"], d["block_table"], d["q"], d["k_pages"], d["v_pages"],
                            o, ws, parent=d.get("parent"), lse=lse, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    ref, ref_lse, tol, lse_tol = R.attention(inp, device="cuda")
    assert (np.abs(o.cpu().double().numpy() - ref) <= tol).all()
    assert (np.abs(lse.cpu().double().numpy() - ref_lse) <= lse_tol).all()


def test_rotation_into_a_far_pool():
    inp = rope_inputs(M=40, Hq=4, Hkv=2, dh=128, sections=[45], L=2, pad=3, seed=2)
    q, k, v, _ = run_rope(inp, 4, [45], "halves")
    d, to = far_pools(inp, 2 ** 20)
    slot = inp["slot"].long()
    d["slot"] = torch.where(slot >= 0, to[(slot // 16).clamp(min=0)] * 16 + slot % 16, -1).to(torch.int32).cuda()
    cfg = lbx.make_page_cfg(2, 1, 40, 4, 2, 128, 16, 2 ** 20, 1)
    out, status = torch.full_like(q, 77.0).cuda(), status_word()
    lbx.lbx_qk_norm_rope(cfg, lbx.make_rope_cfg([45]), d["qkv"], d["inv_freq"], d["pos"], d["slot"], out, d["k_pages"],
                         d["v_pages"], q_weight=d["q_weight"], k_weight=d["k_weight"], d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and same_bits(out.cpu(), q)
    for got, want in ((d["k_pages"], k), (d["v_pages"], v)):
        assert same_bits(got[:, to.cuda()].cpu(), want)


def test_commit_in_a_far_pool():
    inp = R.make_attention([15, 31, 200], [22, 40, 64], 2, 2, 128, 16, L=2, kind="random", seed=3)
    inp["accepted"] = torch.tensor([20, 39, 63], dtype=torch.int32)
    k, v, out, _ = run_commit(inp)
    d, to = far_pools(inp, 2 ** 20)
    table = inp["block_table"].long()
    d["block_table"] = torch.where(table >= 0, to[table.clamp(min=0)], -1).to(torch.int32).cuda()
    cfg = lbx.make_page_cfg(2, 3, d["parent"].shape[0], 2, 2, 128, 16, 2 ** 20, table.shape[1])
    ctx, status = i32([0] * 3), status_word()
    lbx.lbx_page_commit(cfg, d["start"], d["ctx_len"], d["block_table"], d["parent"], d["accepted"], d["k_pages"],
                        d["v_pages"], ctx, d_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and ctx.tolist() == out
    for got, want in ((d["k_pages"], k), (d["v_pages"], v)):
        assert same_bits(got[:, to.cuda()].cpu(), want)


@pytest.mark.parametrize("dh,new", [(64, 150), (128, 40), (128, 900), (256, 150)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_two_parts_beside_infinities_nan_and_bad_pages(dh, new, dtype):
    inp = R.make_attention([20, 200, 30], [3, new, 40], 8, 2, dh, 16, dtype=dtype, seed=6)
    split = dict(weights=lbx.LBX_WEIGHTS_SPLIT)
    clean, clean_lse, _ = run_split(inp, **split)
    q, k, M = inp["q"], inp["k_pages"], 3 + new + 40
    q[:, 0:3] = q[:, 0:3].abs() + 0.5
    for p in range(23):
        k[:, inp["block_table"][0, p // 16], p % 16] = -torch.inf
    q[0, 3 + new // 2, 1, 5] = torch.nan
    inp["block_table"][2, 1] = inp["k_pages"].shape[1]
    o, lse, status = run_split(inp, **split)
    assert status == lbx.LBX_EINVAL
    assert (o[:, :3] == 0).all() and (lse[:, :3] == -torch.inf).all()
    at = 3 + new // 2
    assert o[0, at, 1].isnan().all() and lse[0, at, 1].isnan()
    same = torch.ones(o.shape[:3], dtype=torch.bool)
    same[:, :3] = same[:, M - 40:] = same[0, at, 1] = False
    assert torch.equal(o[same], clean[same]) and torch.equal(lse[same], clean_lse[same])


def run_split(inp, **kw):
    cfg, d = page_cfg(inp, **kw), {k: None if v is None else v.cuda() for k, v in inp.items()}
    o = torch.full_like(d["q"], 55.0)
    lse, ws, status = torch.full(o.shape[:-1], 55.0, device="cuda"), lbx.new_paged_workspace(cfg), status_word()
    torch.cuda.synchronize()
    lbx.lbx_paged_attention(cfg, d["start"], d["ctx_len"], d["block_table"], d["q"], d["k_pages"], d["v_pages"], o,
                            ws, parent=d["parent"], lse=lse, d_status=status)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), int(status.item())
