"""Softmax weights that meet the values in two 16-bit parts: always for few rows over few
keys, elsewhere where the caller asks for it.

The first part is off by half a step u of a weight at most (2^-8 in bf16, 2^-11 in f16), the
second by half a step of that rest, so that a weight is good to u^2; in f16, where weights are
taken 2^7 times as large, a rest below the normal range adds 2^-25, 2^-32 of the row's largest.
With page_ref's e, the score's error, and its share of a long sum
    |o - o_ref| <= u |o_ref| + (u^2 + 2 e + 2^-20 + far) sum w |v| + [f16] (2^-25 + 2^-32 sum |v|).
One rounding of the weights is far outside of it wherever o is small beside sum w |v|."""
import numpy as np
import pytest
import torch

import page_ref as R
from test_gpu_paged import built, page_cfg, status_word  # noqa: F401
from tree_verify_linear_gb300 import lbx

pytestmark = pytest.mark.gpu

CASES = {
    "few_64": dict(ctx=[300, 7], new=[2, 1], Hq=8, Hkv=2, dh=64, page=16),
    "few_128": dict(ctx=[2000], new=[1], Hq=8, Hkv=2, dh=128, page=64),
    "few_tree": dict(ctx=[300, 0, 127], new=[8, 1, 6], Hq=3, Hkv=3, dh=128, page=16, kind="random"),
    "few_joined": dict(ctx=[9000], new=[1], Hq=6, Hkv=1, dh=256, page=64),
    "few_256": dict(ctx=[500, 90], new=[1, 1], Hq=24, Hkv=4, dh=256, page=64),
}
SPLIT = {
    # single tokens on the tensor-memory path, cut and whole
    "tokens_64": dict(ctx=[9000, 7001, 5], new=[1] * 3, Hq=16, Hkv=4, dh=64, page=16),
    "tokens_128": dict(ctx=[9000, 7001, 5], new=[1] * 3, Hq=16, Hkv=4, dh=128, page=32),
    "tokens_256": dict(ctx=[9000, 7001, 5], new=[1] * 3, Hq=16, Hkv=4, dh=256, page=64),
    "group_of_12": dict(ctx=[100, 33], new=[1, 1], Hq=24, Hkv=2, dh=128, page=16),
    # trees and short chunks
    "tree_64": dict(ctx=[700, 90], new=[22, 40], Hq=8, Hkv=2, dh=64, page=32, kind="random"),
    "tree_128": dict(ctx=[700, 90], new=[22, 64], Hq=8, Hkv=2, dh=128, page=32, kind="random"),
    "tree_128_wide": dict(ctx=[300, 90], new=[64, 64], Hq=32, Hkv=2, dh=128, page=16, kind="random"),
    "tree_256": dict(ctx=[700, 90], new=[22, 64], Hq=12, Hkv=2, dh=256, page=64, kind="random"),
    "chunk_64": dict(ctx=[400], new=[64], Hq=6, Hkv=2, dh=64, page=64),
    "chunk_256": dict(ctx=[400, 0], new=[64, 33], Hq=6, Hkv=2, dh=256, page=64),
    # longer ones, with 768 rows of a request and more at head dimension 128 too
    "ragged": dict(ctx=[300, 200, 50], new=[1, 300, 22], Hq=8, Hkv=2, dh=128, page=32),
    "prompts_64": dict(ctx=[0, 100], new=[300, 77], Hq=4, Hkv=2, dh=64, page=16),
    "prompts_128_wide": dict(ctx=[0, 60], new=[500, 401], Hq=8, Hkv=2, dh=128, page=32, L=2),
    "prompts_256": dict(ctx=[0, 100], new=[300, 77], Hq=4, Hkv=2, dh=256, page=64, pad=3),
}


def magnitudes(inp, device):
    """sum w |v| of each output: the attention of |v|."""
    return R.attention(dict(inp, v_pages=inp["v_pages"].abs()), device=device)[0]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_weights_of_few_rows_have_two_parts(name, dtype):
    check(R.make_attention(**CASES[name], dtype=dtype, seed=300 + len(name)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(SPLIT))
def test_weights_have_two_parts_where_asked_for(name, dtype):
    check(R.make_attention(**SPLIT[name], dtype=dtype, seed=300 + len(name)), dtype,
          weights=lbx.LBX_WEIGHTS_SPLIT)


def check(inp, dtype, **kw):
    cfg = page_cfg(inp, **kw)
    d = {k: None if v is None else v.cuda() for k, v in inp.items()}
    o, ws, status = torch.full_like(d["q"], 55.0), lbx.new_paged_workspace(cfg), status_word()
    torch.cuda.synchronize()
    for _ in range(2):
        lbx.lbx_paged_attention(cfg, d["start"], d["ctx_len"], d["block_table"], d["q"], d["k_pages"],
                                d["v_pages"], o, ws, parent=d["parent"], d_status=status)
    torch.cuda.synchronize()
    o = o.cpu()
    assert int(status.item()) == 0
    ref, ref_lse, _, lse_tol = R.attention(inp, device="cuda")
    size, u = magnitudes(inp, "cuda"), R.U[inp["q"].dtype]
    start = inp["start"].tolist()
    assert (o[:, start[-1]:] == 55.0).all()
    most = float(inp["v_pages"][~inp["v_pages"].isnan()].abs().max())
    for b, t in enumerate(inp["ctx_len"].tolist()):
        at, n = slice(start[b], start[b + 1]), start[b + 1] - start[b]
        far = (t + n) * 2.0 ** -24 if t + n > 4096 else 0.0
        e = lse_tol[:, at, :, None] - 2.0 ** -20 * (1 + np.abs(ref_lse[:, at, :, None])) - far
        tol = u * np.abs(ref[:, at]) + (u * u + 2 * e + 2.0 ** -20 + far) * size[:, at]
        if dtype == "f16":
            tol += 2.0 ** -25 + 2.0 ** -32 * (t + n) * most
        over = np.abs(o[:, at].double().numpy() - ref[:, at]) / (1.02 * tol)
        assert np.isfinite(over).all() and over.max() <= 1, (b, float(over.max()))
