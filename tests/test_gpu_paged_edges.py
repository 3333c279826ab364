"""GPU parity of the paged cache's operators at the edges of their paths: lists of as
many pieces as one call joins, values that are not finite, angles far below one.  The
bounds are page_ref's unless a test derives its own."""
import numpy as np
import pytest
import torch

import page_ref as R
from test_gpu_paged import (built, check_attention, page_cfg, rope_inputs, run_attention,  # noqa: F401
                            run_rope, status_word)
from tree_verify_linear_gb300 import lbx

pytestmark = pytest.mark.gpu


# ---- few rows over the longest list that their path takes -------------------------

def longest(pieces_off=9, dh=64, **kw):
    """One request of one layer and KV head with two units of 128 keys per CTA, less
    `pieces_off`: the most pieces that few rows join."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    units = 2 * (sms // 2 * 2) - pieces_off
    return units, R.make_attention([128 * units - 5], [1], 4, 1, dh, 16, seed=21, **kw)


@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("off", [0, 9])
def test_one_token_over_the_longest_list_of_few_rows(dh, off):
    check_attention(longest(off, dh)[1], device="cuda", calls=2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pieces_of_minus_infinity_among_the_most(dtype):
    """Units of keys whose scores are all -inf, at both ends of the list: the row is that of a
    request without them."""
    units, inp = longest(dtype=dtype)
    inp["q"] = inp["q"].abs() + 0.5
    dead = list(range(0, 3)) + list(range(units // 2, units - 1))
    pages = [8 * u + j for u in dead for j in range(8)]
    alive = [p for p in range(8 * units) if p not in set(pages)]
    table = inp["block_table"]
    inp["k_pages"][:, table[0, pages].long()] = -torch.inf
    o, lse, status = run_attention(inp, calls=2)
    assert status == 0
    ref, ref_lse, tol, lse_tol = R.attention(
        dict(inp, block_table=table[:, alive], ctx_len=inp["ctx_len"] - 128 * len(dead)), device="cuda")
    assert (np.abs(o.double().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().numpy() - ref_lse) <= lse_tol).all()


def test_pages_outside_the_pool_among_the_most_pieces():
    """They are reported, and the workspace serves the next call."""
    units, inp = longest()
    cfg, d = page_cfg(inp), {k: None if v is None else v.cuda() for k, v in inp.items()}
    ws, status, o = lbx.new_paged_workspace(cfg), status_word(), torch.zeros_like(d["q"])
    bad = d["block_table"].clone()
    bad[0, 8 * (units // 2):8 * (units - 1)] = -1
    torch.cuda.synchronize()
    for table in (bad, d["block_table"]):
        lbx.lbx_paged_attention(cfg, d["start"], d["ctx_len"], table, d["q"], d["k_pages"], d["v_pages"], o, ws,
                                d_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == (lbx.LBX_EINVAL if table is bad else 0)
        status.zero_()
    ref, _, tol, _ = R.attention(inp, device="cuda")
    assert (np.abs(o.cpu().double().numpy() - ref) <= tol).all()


# ---- dimensions that do not turn ---------------------------------------------------

ODD = [torch.inf, -torch.inf, torch.nan, -0.0]


@pytest.mark.parametrize("pairing,dh,half", [("adjacent", 64, 3), ("adjacent", 128, 37), ("adjacent", 256, 64),
                                             ("halves", 64, 3), ("halves", 128, 45), ("halves", 256, 5),
                                             ("halves", 128, 16), ("halves", 64, 0), ("adjacent", 64, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dimensions_that_do_not_turn_stay(pairing, dh, half, dtype):
    """Without a norm the dimensions past the last pair are the input's, whatever stands beside
    them; and what turns does not see them."""
    inp = rope_inputs(M=24, Hq=4, Hkv=2, dh=dh, sections=[half], dtype=dtype, norm=False, seed=5)
    clean = run_rope(inp, 4, [half], pairing)
    rng = np.random.default_rng(6)
    x = inp["qkv"]
    for i in range(2 * half, dh):
        at = torch.from_numpy(rng.random(x.shape[:3]) < 0.3)
        x[..., i][at] = ODD[i % 4]
    q, k, _, status = run_rope(inp, 4, [half], pairing)
    assert status == 0
    slot = inp["slot"].long()
    for got, was, came in ((q, clean[0], x[:, :, :4]),
                           (k.flatten(1, 2)[:, slot], clean[1].flatten(1, 2)[:, slot], x[:, :, 4:6])):
        assert torch.equal(got[..., :2 * half], was[..., :2 * half])
        rest, want = got[..., 2 * half:], came[..., 2 * half:]
        number = ~want.isnan()
        assert torch.equal(rest.isnan(), ~number)
        assert torch.equal(rest[number].view(torch.int16), want[number].view(torch.int16))


# ---- small angles ------------------------------------------------------------------

@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("half", [32, 29])
def test_angles_far_below_one_keep_their_digits(pairing, dtype, half):
    """One value of a pair is 0, so that the other one's sine stands alone: it is off by 16 2^-24
    of itself (the frequency's fraction of a turn to 2^-24, its product, the conversion, pi, the
    sine, the product) and the rounding of the result, in f16 half a step of 2^-24 at most."""
    M, dh = 16, 64
    inp = rope_inputs(M=M, Hq=2, Hkv=1, dh=dh, sections=[half], dtype=dtype, norm=False)
    inp["inv_freq"] = (10.0 ** (-3 - 6 * torch.arange(half).double() / (half - 1))).float()
    inp["pos"][0] = torch.tensor([1, -1, 2, -2, 3, -3, 5, -5, 7, -7, 100, -100, 1001, -1001, 4000, -4000],
                                 dtype=torch.int32)
    first = torch.arange(half) if pairing == "halves" else 2 * torch.arange(half)
    second = first + (half if pairing == "halves" else 1)
    for zero, one, sign in ((first, second, -1.0), (second, first, 1.0)):
        x = inp["qkv"]
        x[..., one], x[..., zero] = 1.5, 0.0
        q, k, _, status = run_rope(inp, 2, [half], pairing)
        assert status == 0
        t = inp["pos"][0].double()[:, None] * inp["inv_freq"].double()
        ref = sign * 1.5 * torch.sin(t)
        u = R.U[R.DTYPE[dtype]]
        tol = (u + 17 * 2.0 ** -24) * ref.abs() + (2.0 ** -25 if dtype == "f16" else 0.0)
        for got in (q[0], k.flatten(1, 2)[0, inp["slot"].long()]):
            off = (got[..., zero].double() - ref[:, None]).abs() / tol[:, None]
            assert off.max() <= 1, float(off.max())
