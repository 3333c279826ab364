"""Few rows over few keys: their softmax weights meet the values in two 16-bit parts.

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
from test_gpu_paged import built, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = {
    "few_64": dict(ctx=[300, 7], new=[2, 1], Hq=8, Hkv=2, dh=64, page=16),
    "few_128": dict(ctx=[2000], new=[1], Hq=8, Hkv=2, dh=128, page=64),
    "few_tree": dict(ctx=[300, 0, 127], new=[8, 1, 6], Hq=3, Hkv=3, dh=128, page=16, kind="random"),
    "few_joined": dict(ctx=[9000], new=[1], Hq=6, Hkv=1, dh=256, page=64),
    "few_256": dict(ctx=[500, 90], new=[1, 1], Hq=24, Hkv=4, dh=256, page=64),
}


def magnitudes(inp, device):
    """sum w |v| of each output: the attention of |v|."""
    return R.attention(dict(inp, v_pages=inp["v_pages"].abs()), device=device)[0]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_weights_have_two_parts(name, dtype):
    inp = R.make_attention(**CASES[name], dtype=dtype, seed=300 + len(name))
    o, _, status = run_attention(inp)
    assert status == 0
    ref, ref_lse, _, lse_tol = R.attention(inp, device="cuda")
    size, u = magnitudes(inp, "cuda"), R.U[inp["q"].dtype]
    start = inp["start"].tolist()
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
