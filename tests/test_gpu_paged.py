"""GPU parity of the paged cache's operators with their definitions in 64 bits,
through the C ABI.  The error bounds are derived in page_ref; whole numbers, moved
rows and everything that must stay untouched compare equal."""
import numpy as np
import pytest
import torch

import page_ref as R
from tree_verify_linear_gb300 import lbx

pytestmark = pytest.mark.gpu
TYPE = {torch.bfloat16: lbx.LBX_BF16, torch.float16: lbx.LBX_F16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for -m gpu tests")
    from tree_verify_linear_gb300 import build
    build.build()
    lbx.load()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def i32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


# ---- block tables ---------------------------------------------------------------

def tables_case(ctx, new, page, held=None, pad=0, seed=0, spare=5):
    rng = np.random.default_rng(seed)
    want = [R.pages_of(t + n, page) for t, n in zip(ctx, new)]
    held = [R.pages_of(t, page) for t in ctx] if held is None else held
    n_pages = sum(max(h, w) for h, w in zip(held, want)) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    width = max(want + held) + 1
    table, at = np.full((len(ctx), width), -9, dtype=np.int32), 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    stack = np.full(n_pages, -9, dtype=np.int32)
    stack[:n_pages - at] = order[at:]
    return dict(ctx=ctx, new=new, held=held, n_free=n_pages - at, table=table, stack=stack, page=page,
                M=max(1, sum(new) + pad))


def run_tables(c, M=None, n_free=None, calls=1, stream=None):
    M = c["M"] if M is None else M
    B, width = c["table"].shape
    cfg = lbx.make_page_cfg(1, B, M, 1, 1, 64, c["page"], len(c["stack"]), width)
    d = {"block_table": i32(c["table"]), "free_list": i32(c["stack"]), "held_out": i32([-3] * B),
         "n_free_out": i32([-3]), "start": i32([-3] * (B + 1)), "slot": i32([-3] * M), "pos": i32([-3] * M)}
    ins = [i32(c["ctx"]), i32(c["new"]), i32(c["held"]), i32([c["n_free"] if n_free is None else n_free])]
    status = status_word()
    torch.cuda.synchronize()
    for _ in range(calls):
        lbx.lbx_page_tables(cfg, *ins, d["block_table"], d["free_list"], d["held_out"], d["n_free_out"],
                            d["start"], d["slot"], d["pos"], d_status=status, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in d.items()}, int(status.item())


def many(n, seed, page):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, 40 * page, n).tolist()
    new = (rng.integers(0, 4, n) * rng.integers(0, 3 * page, n)).tolist()
    held = [max(0, R.pages_of(t, page) + int(x)) for t, x in zip(ctx, rng.integers(0, 3, n))]
    for b in rng.integers(0, n, n // 6):
        ctx[b] = new[b] = 0
    return ctx, new, held


TABLES = {
    "one_token": dict(ctx=[0], new=[1], page=16),
    "nothing": dict(ctx=[0, 5], new=[0, 0], page=16, pad=3),
    "page_runs_full": dict(ctx=[15, 16, 17, 31], new=[1, 1, 1, 1], page=16),
    "prompt_and_decode": dict(ctx=[0, 100, 0], new=[1000, 1, 257], page=64, pad=9),
    "ended_requests_feed_others": dict(ctx=[0, 640, 0, 0], new=[0, 1, 0, 500], page=32,
                                       held=[9, 20, 4, 0], spare=3),
    "rejected_drafts": dict(ctx=[63, 64, 65], new=[1, 0, 22], page=64, held=[3, 2, 2]),
    "big_pages": dict(ctx=[255, 256, 1], new=[2, 0, 255], page=256, pad=1),
    "requests_300": dict(zip(("ctx", "new", "held"), many(300, 1, 16)), page=16, pad=40),
    "requests_513": dict(zip(("ctx", "new", "held"), many(513, 2, 64)), page=64),
    "requests_2048": dict(zip(("ctx", "new", "held"), many(2048, 3, 16)), page=16, pad=3),
}


@pytest.mark.parametrize("name", sorted(TABLES))
@pytest.mark.parametrize("calls", [1, 2])
def test_tables(name, calls):
    c = tables_case(**TABLES[name])
    got, status = run_tables(c, calls=calls)
    assert status == 0
    want = R.tables(c["ctx"], c["new"], c["held"], c["n_free"], c["table"], c["stack"], c["page"], c["M"])
    for k, v in want.items():
        assert np.array_equal(got[k], np.asarray(v)), k


def test_tables_that_take_every_page():
    c = tables_case([0, 40], [100, 30], 16, spare=0)
    got, status = run_tables(c)
    assert status == 0 and got["n_free_out"][0] == 0


BAD_TABLES = {
    "too_few_pages": (dict(ctx=[0, 40], new=[100, 30]), dict(n_free=3), lbx.LBX_EPAGES),
    "more_tokens_than_rows": (dict(ctx=[0, 40], new=[100, 30]), dict(M=129), lbx.LBX_EINVAL),
    "negative_length": (dict(ctx=[0, 40], new=[100, 30], set=("ctx", 1, -1)), {}, lbx.LBX_EINVAL),
    "negative_new": (dict(ctx=[0, 40], new=[100, 30], set=("new", 0, -1)), {}, lbx.LBX_EINVAL),
    "negative_held": (dict(ctx=[0, 40], new=[100, 30], set=("held", 0, -1)), {}, lbx.LBX_EINVAL),
    "held_past_the_table": (dict(ctx=[0, 40], new=[100, 30], set=("held", 0, 99)), {}, lbx.LBX_EINVAL),
    "longer_than_the_table": (dict(ctx=[0, 40], new=[100, 30], set=("ctx", 1, 2 ** 30)), {}, lbx.LBX_EINVAL),
    "length_sum_past_32_bits": (dict(ctx=[0, 40], new=[100, 30], set=("ctx", 1, 2 ** 31 - 5)), {},
                                lbx.LBX_EINVAL),
    "negative_stack": (dict(ctx=[0, 40], new=[100, 30]), dict(n_free=-1), lbx.LBX_EINVAL),
    "stack_would_outgrow_the_pool": (dict(ctx=[0, 0], new=[0, 0], held=[3, 3]), dict(n_free=8), lbx.LBX_EINVAL),
}


@pytest.mark.parametrize("name", sorted(BAD_TABLES))
def test_bad_batches_write_no_tables(name):
    case, how, code = BAD_TABLES[name]
    case = dict(case)
    change = case.pop("set", None)
    c = tables_case(page=16, **case)
    if change:
        c[change[0]] = list(c[change[0]])
        c[change[0]][change[1]] = change[2]
    got, status = run_tables(c, **how)
    assert status == code
    assert np.array_equal(got["block_table"], c["table"]) and np.array_equal(got["free_list"], c["stack"])
    for k in ("held_out", "n_free_out", "start", "slot", "pos"):
        assert (got[k] == -3).all(), k


def test_a_page_outside_the_pool_gives_no_slot():
    c = tables_case([20, 20], [3, 3], 16)
    c["table"][1, 1] = len(c["stack"])
    got, status = run_tables(c)
    assert status == lbx.LBX_EINVAL
    assert (got["slot"][3:6] == -1).all() and (got["slot"][:3] >= 0).all()


# ---- norms and rotation ----------------------------------------------------------

def rope_inputs(M, Hq, Hkv, dh, sections, L=1, dtype="bf16", page=16, far=5000, pad=0, seed=0, base=1e4,
                norm=True):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, half = R.DTYPE[dtype], sum(sections)
    n_pages = R.pages_of(M, page) + 2
    slot = rng.permutation(n_pages * page)[:M].astype(np.int32)
    if pad:
        slot[rng.permutation(M)[:pad]] = -1
    return {"qkv": (torch.randn(L, M, Hq + 2 * Hkv, dh, generator=g) * 3).to(dt),
            "q_weight": torch.randn(L, dh, generator=g) if norm else None,
            "k_weight": torch.randn(L, dh, generator=g) if norm else None,
            "inv_freq": (base ** (-torch.arange(half).double() / max(half, 1))).float(),
            "pos": torch.from_numpy(rng.integers(0, far, (len(sections), M)).astype(np.int32)),
            "slot": torch.from_numpy(slot),
            "k_pages": torch.randn(L, n_pages, page, Hkv, dh, generator=g).to(dt),
            "v_pages": torch.randn(L, n_pages, page, Hkv, dh, generator=g).to(dt)}


def run_rope(inp, Hq, sections, pairing, eps=1e-6, stream=None):
    L, M, H, dh = inp["qkv"].shape
    n_pages, page, Hkv = inp["k_pages"].shape[1:4]
    cfg = lbx.make_page_cfg(L, 1, M, Hq, Hkv, dh, page, n_pages, 1, dtype=TYPE[inp["qkv"].dtype])
    rc = lbx.make_rope_cfg(sections, eps=eps, pairing=lbx.LBX_ROPE_HALVES if pairing == "halves"
                           else lbx.LBX_ROPE_ADJACENT)
    d = {k: None if v is None else v.cuda() for k, v in inp.items()}
    q = torch.full((L, M, Hq, dh), 77.0, dtype=inp["qkv"].dtype, device="cuda")
    status = status_word()
    torch.cuda.synchronize()
    lbx.lbx_qk_norm_rope(cfg, rc, d["qkv"], d["inv_freq"] if sum(sections) else None, d["pos"], d["slot"],
                         q, d["k_pages"], d["v_pages"], q_weight=d["q_weight"], k_weight=d["k_weight"],
                         d_status=status, stream=stream)
    torch.cuda.synchronize()
    return q.cpu(), d["k_pages"].cpu(), d["v_pages"].cpu(), int(status.item())


def check_rope(inp, Hq, sections, pairing, eps=1e-6, skipped=()):
    q, k, v, status = run_rope(inp, Hq, sections, pairing, eps)
    L, M, H, dh = inp["qkv"].shape
    Hkv, u = inp["k_pages"].shape[3], R.U[inp["qkv"].dtype]
    slot = inp["slot"].long().clone()
    slot[list(skipped)] = -1
    on = slot >= 0
    kr, vr = inp["k_pages"].flatten(1, 2).clone(), inp["v_pages"].flatten(1, 2).clone()
    for l in range(L):
        for name, lo, hi, got in (("q_weight", 0, Hq, q[l]),
                                  ("k_weight", Hq, Hq + Hkv, k.flatten(1, 2)[l])):
            w = None if inp[name] is None else inp[name][l]
            ref, tol = R.rope(inp["qkv"][l, :, lo:hi], w, inp["inv_freq"], inp["pos"], sections, pairing, eps)
            got = got[on] if name == "q_weight" else got[slot[on]]
            at = on.numpy()
            over = np.abs(got.double().numpy() - ref[at]) / (u * np.abs(ref[at]) + tol[at] + 2.0 ** -25)
            assert np.isfinite(over).all() and over.max() <= 1, (name, float(over.max()))
        vr[l, slot[on]] = inp["qkv"][l, on, Hq + Hkv:]
    assert torch.equal(v.flatten(1, 2), vr)
    # what no row names stays, bit for bit
    rest = torch.ones(kr.shape[1], dtype=torch.bool)
    rest[slot[on]] = False
    assert torch.equal(k.flatten(1, 2)[:, rest], kr[:, rest])
    assert (q[:, ~on] == 77.0).all()
    return status


ROPE = {
    "one_row": (dict(M=1, Hq=1, Hkv=1, dh=64), [32], "halves"),
    "partial_256": (dict(M=7, Hq=24, Hkv=4, dh=256, L=2), [32], "halves"),
    "whole_128": (dict(M=33, Hq=8, Hkv=2, dh=128, dtype="f16"), [64], "halves"),
    "odd_pairs": (dict(M=19, Hq=3, Hkv=1, dh=128), [5], "halves"),
    "one_pair": (dict(M=5, Hq=3, Hkv=3, dh=64), [1], "adjacent"),
    "odd_pairs_adjacent": (dict(M=19, Hq=3, Hkv=1, dh=256, dtype="f16"), [37], "adjacent"),
    "no_pairs": (dict(M=6, Hq=4, Hkv=2, dh=64), [0], "halves"),
    "no_norm": (dict(M=21, Hq=4, Hkv=2, dh=128, norm=False), [64], "adjacent"),
    "three_axes": (dict(M=50, Hq=5, Hkv=5, dh=128, far=40000), [16, 24, 24], "halves"),
    "four_axes_one_empty": (dict(M=50, Hq=6, Hkv=1, dh=64, dtype="f16"), [7, 0, 3, 11], "adjacent"),
    "padding": (dict(M=100, Hq=6, Hkv=2, dh=64, pad=41), [16], "halves"),
    "far_positions": (dict(M=64, Hq=2, Hkv=1, dh=128, far=2 ** 31 - 1, base=1e7), [64], "halves"),
    "rows_1300": (dict(M=1301, Hq=7, Hkv=1, dh=64, pad=3), [20], "halves"),
    "rows_5000": (dict(M=5003, Hq=2, Hkv=1, dh=256, L=2, page=64), [64], "adjacent"),
    "rows_20000": (dict(M=20011, Hq=3, Hkv=1, dh=64, page=256, dtype="f16"), [8, 8, 8], "halves"),
}


@pytest.mark.parametrize("name", sorted(ROPE))
def test_rope(name):
    sizes, sections, pairing = ROPE[name]
    assert check_rope(rope_inputs(**sizes, sections=sections, seed=len(name)), sizes["Hq"], sections, pairing) == 0


def test_rope_of_negative_positions_and_zero_rows():
    inp = rope_inputs(M=9, Hq=2, Hkv=1, dh=64, sections=[32])
    inp["pos"][0] = torch.arange(-4, 5, dtype=torch.int32) * 1001
    inp["qkv"][:, 3] = 0
    assert check_rope(inp, 2, [32], "halves") == 0


def test_rope_reports_and_skips_a_slot_outside_the_pool():
    inp = rope_inputs(M=9, Hq=2, Hkv=1, dh=64, sections=[32])
    inp["slot"][4] = inp["k_pages"].shape[1] * 16
    assert check_rope(inp, 2, [32], "halves", skipped=[4]) == lbx.LBX_EINVAL


# ---- attention -----------------------------------------------------------------

def page_cfg(inp, **kw):
    L, M, Hq, dh = inp["q"].shape
    n_pages, page, Hkv = inp["k_pages"].shape[1:4]
    return lbx.make_page_cfg(L, len(inp["ctx_len"]), M, Hq, Hkv, dh, page, n_pages,
                             inp["block_table"].shape[1], dtype=TYPE[inp["q"].dtype], **kw)


def run_attention(inp, calls=1, stream=None, want_lse=True, **kw):
    cfg = page_cfg(inp, **kw)
    d = {k: None if v is None else v.cuda() for k, v in inp.items()}
    o = torch.full_like(d["q"], 55.0)
    lse = torch.full(o.shape[:-1], 55.0, device="cuda") if want_lse else None
    ws, status = lbx.new_paged_workspace(cfg), status_word()
    torch.cuda.synchronize()
    for _ in range(calls):
        lbx.lbx_paged_attention(cfg, d["start"], d["ctx_len"], d["block_table"], d["q"], d["k_pages"],
                                d["v_pages"], o, ws, parent=d["parent"], lse=lse, d_status=status,
                                stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), None if lse is None else lse.cpu(), int(status.item())


def check_attention(inp, device="cpu", calls=1, **kw):
    o, lse, status = run_attention(inp, calls=calls, **kw)
    assert status == 0
    live = int(inp["start"][-1])
    assert (o[:, live:] == 55.0).all() and (lse[:, live:] == 55.0).all()
    ref_o, ref_lse, o_tol, lse_tol = R.attention(inp, device=device, **kw)
    over = np.abs(o.double().numpy() - ref_o)[:, :live] / o_tol[:, :live]
    assert np.isfinite(over).all() and over.max(initial=0) <= 1, float(over.max())
    over = np.abs(lse.double().numpy() - ref_lse)[:, :live] / lse_tol[:, :live]
    assert np.isfinite(over).all() and over.max(initial=0) <= 1, float(over.max())
    return o, lse


ATTN = {
    "one_token_alone": dict(ctx=[0], new=[1], Hq=1, Hkv=1, dh=64, page=16),
    "one_token": dict(ctx=[1, 0, 15, 16, 17], new=[1] * 5, Hq=4, Hkv=2, dh=128, page=16),
    "one_token_256": dict(ctx=[2000, 63, 64], new=[1] * 3, Hq=24, Hkv=4, dh=256, page=64),
    "one_token_f16": dict(ctx=[700, 0], new=[1, 1], Hq=8, Hkv=1, dh=64, page=32, dtype="f16", pad=3),
    "chunk_of_two": dict(ctx=[5], new=[2], Hq=2, Hkv=2, dh=64, page=16),
    "prompts": dict(ctx=[0, 0, 0], new=[127, 128, 129], Hq=4, Hkv=2, dh=128, page=16, pad=2),
    "prompts_64": dict(ctx=[0, 0], new=[257, 31], Hq=3, Hkv=1, dh=64, page=256),
    "prompts_256": dict(ctx=[0, 0, 0], new=[100, 1, 260], Hq=6, Hkv=1, dh=256, page=64),
    "chunk": dict(ctx=[300, 1], new=[70, 200], Hq=6, Hkv=2, dh=256, page=32, L=2),
    "chunk_f16": dict(ctx=[129, 513], new=[65, 300], Hq=8, Hkv=2, dh=128, page=128, dtype="f16"),
    "chunks_and_decode": dict(ctx=[0, 1000, 77, 400, 9], new=[90, 1, 0, 1, 33], Hq=4, Hkv=1, dh=64,
                              page=64, pad=7),
    "requests_without_tokens": dict(ctx=[0, 5, 9], new=[0, 0, 3], Hq=2, Hkv=1, dh=128, page=16),
    "no_tokens": dict(ctx=[0, 5], new=[0, 0], Hq=2, Hkv=1, dh=128, page=16, pad=4),
    "group_of_7": dict(ctx=[50], new=[90], Hq=14, Hkv=2, dh=64, page=16, dtype="f16"),
    "group_of_48": dict(ctx=[70, 3], new=[5, 9], Hq=48, Hkv=1, dh=128, page=32),
    "group_of_128": dict(ctx=[70, 3], new=[5, 1], Hq=128, Hkv=1, dh=256, page=32),
    "group_of_100": dict(ctx=[70, 3], new=[5, 1], Hq=100, Hkv=1, dh=64, page=32, dtype="f16"),
    "many_heads": dict(ctx=[33, 64], new=[3, 1], Hq=40, Hkv=40, dh=64, page=16),
    "wide_scores": dict(ctx=[400, 300], new=[6, 70], Hq=4, Hkv=2, dh=256, page=64, width=20.0),
    "wide_scores_f16": dict(ctx=[400], new=[140], Hq=4, Hkv=2, dh=64, page=64, width=20.0, dtype="f16"),
    "tree": dict(ctx=[100, 0, 64], new=[22, 22, 7], Hq=24, Hkv=4, dh=256, page=64, kind="random", L=2),
    "tree_chain": dict(ctx=[64], new=[64], Hq=2, Hkv=1, dh=128, page=16, kind="chain"),
    "tree_star": dict(ctx=[63, 1], new=[64, 2], Hq=8, Hkv=1, dh=64, page=32, kind="star", dtype="f16"),
    "tree_wide": dict(ctx=[130, 500], new=[64, 1], Hq=16, Hkv=2, dh=128, page=256, kind="random", pad=5),
    "tree_of_some": dict(ctx=[13, 7, 29], new=[5, 0, 40], Hq=6, Hkv=3, dh=256, page=16, kind="random"),
    "tree_one_token": dict(ctx=[0, 200], new=[1, 1], Hq=6, Hkv=1, dh=256, page=16, kind="random", dtype="f16"),
}


@pytest.mark.parametrize("name", sorted(ATTN))
def test_attention(name):
    check_attention(R.make_attention(**ATTN[name], seed=700 + len(name)))


# Enough keys that every CTA walks many blocks and tiles, whole ones and cut ones.
BUSY = {
    "decode_long_64": dict(ctx=[20000, 3], new=[1, 1], Hq=8, Hkv=1, dh=64, page=16),
    "decode_long_128_f16": dict(ctx=[9000, 7000, 1], new=[1] * 3, Hq=16, Hkv=2, dh=128, page=16, dtype="f16"),
    "decode_long_256": dict(ctx=[9001, 4000], new=[1, 1], Hq=12, Hkv=2, dh=256, page=64),
    "tree_long_256": dict(ctx=[6000, 2501], new=[22, 22], Hq=12, Hkv=2, dh=256, page=64, kind="random", L=2),
    "tree_long_128": dict(ctx=[7000], new=[40], Hq=7, Hkv=1, dh=128, page=32, kind="random", dtype="f16"),
    "chunk_long_128": dict(ctx=[3000, 0, 40], new=[700, 1500, 1], Hq=8, Hkv=2, dh=128, page=32),
    "chunk_long_256": dict(ctx=[2500, 10], new=[601, 900], Hq=12, Hkv=2, dh=256, page=16, pad=3),
    "chunk_long_256_f16": dict(ctx=[100], new=[1800], Hq=8, Hkv=2, dh=256, page=128, dtype="f16"),
    "chunk_long_64": dict(ctx=[4000, 0], new=[1000, 2100], Hq=6, Hkv=2, dh=64, page=64),
    "layers": dict(ctx=[800, 333, 0], new=[1, 300, 77], Hq=8, Hkv=4, dh=128, page=64, L=5),
    "requests_700": dict(ctx=[(13 * b) % 170 for b in range(700)], new=[(b * 7) % 4 for b in range(700)],
                         Hq=12, Hkv=2, dh=64, page=16),
    "requests_500_of_256": dict(ctx=[(29 * b) % 300 for b in range(500)],
                                new=[40 if b % 50 == 3 else b % 2 for b in range(500)], Hq=4, Hkv=2, dh=256,
                                page=32, pad=9),
    "trees_of_400": dict(ctx=[(31 * b) % 200 for b in range(400)], new=[(b * 11) % 23 for b in range(400)],
                         Hq=4, Hkv=1, dh=128, page=16, kind="random"),
    "wide_batch": dict(ctx=[(37 * b) % 900 for b in range(150)], new=[1] * 150, Hq=8, Hkv=2, dh=128, page=16),
}


@pytest.mark.parametrize("name", sorted(BUSY))
def test_long_ragged_batches(name):
    check_attention(R.make_attention(**BUSY[name], seed=800 + len(name)), device="cuda", calls=2)


def test_without_lse_and_another_scale():
    inp = R.make_attention([40, 3], [9, 30], 4, 2, 128, 16, seed=5)
    o, _, status = run_attention(inp, want_lse=False, scale=0.3)
    ref, _, tol, _ = R.attention(inp, scale=0.3)
    assert status == 0 and (np.abs(o.double().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("dh,dtype", [(64, "f16"), (128, "bf16"), (256, "bf16")])
def test_scores_of_minus_infinity_and_nan(dh, dtype):
    """A row that sees only keys of -inf gets 0 and -inf; one NaN among its scores
    makes a row NaN; other rows, other requests do not change."""
    inp = R.make_attention([20, 200, 30], [3, 150, 40], 2, 1, dh, 16, dtype=dtype, seed=6)
    clean, clean_lse, _ = run_attention(inp)
    q, k = inp["q"], inp["k_pages"]
    q[:, 0:3] = q[:, 0:3].abs() + 0.5  # request 0: every score -inf
    for p in range(23):
        k[:, inp["block_table"][0, p // 16], p % 16] = -torch.inf
    q[0, 3 + 70, 1, 5] = torch.nan  # request 1, token 70: one head's scores are NaN
    o, lse, status = run_attention(inp)
    assert status == 0
    assert (o[:, :3] == 0).all() and (lse[:, :3] == -torch.inf).all()
    assert o[0, 73, 1].isnan().all() and lse[0, 73, 1].isnan()
    same = torch.ones(q.shape[1], dtype=torch.bool)
    same[:3] = same[73] = False
    assert torch.equal(o[:, same], clean[:, same]) and torch.equal(lse[:, same], clean_lse[:, same])
    assert torch.equal(o[0, 73, 0], clean[0, 73, 0])


def test_some_scores_of_minus_infinity():
    """Keys of -inf beside others take no weight, first blocks of nothing else included."""
    inp = R.make_attention([300], [20], 2, 1, 128, 16, seed=7)
    inp["q"] = inp["q"].abs() + 0.5
    for p in list(range(0, 140)) + [200, 305]:
        inp["k_pages"][:, inp["block_table"][0, p // 16], p % 16] = -torch.inf
    o, lse, status = run_attention(inp)
    keep = inp["k_pages"].clone()
    keep[keep == -torch.inf] = -1000.0  # exp of what is left is 0 as well
    ref, ref_lse, tol, lse_tol = R.attention(dict(inp, k_pages=keep))
    assert status == 0 and (np.abs(o.double().numpy() - ref) <= tol + 1e-3).all()
    assert np.isfinite(lse.numpy()).all()


def bad_attention(change):
    inp = R.make_attention([40, 7], [9, 30], 4, 2, 64, 16, kind="random", seed=9)
    change(inp)
    return run_attention(inp)


BAD = {
    "first_not_zero": lambda i: i["start"].__setitem__(0, 1),
    "start_falls": lambda i: i["start"].__setitem__(1, 40),
    "past_the_rows": lambda i: i["start"].__setitem__(2, 40),
    "negative_length": lambda i: i["ctx_len"].__setitem__(0, -1),
    "past_the_table": lambda i: i["ctx_len"].__setitem__(1, 16 * i["block_table"].shape[1] - 29),
    "root_has_a_parent": lambda i: i["parent"].__setitem__(9, 0),
    "parent_not_before": lambda i: i["parent"].__setitem__(5, 5),
    "second_root": lambda i: i["parent"].__setitem__(3, -1),
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_bad_batches_write_no_outputs(name):
    o, lse, status = bad_attention(BAD[name])
    assert status == lbx.LBX_ETREE and (o == 55.0).all() and (lse == 55.0).all()


WILD = [(2 ** 31 - 1, -2 ** 31), (1_800_000_000, -1_800_000_000), (2 ** 30, -2 ** 31), (-2 ** 31, 2 ** 31 - 1),
        (2 ** 31 - 1, 2 ** 31 - 1), (-1, -2 ** 31)]


@pytest.mark.parametrize("first,second", WILD)
def test_starts_whose_differences_wrap_are_refused(first, second):
    def change(inp):
        inp["start"][1], inp["start"][2] = first, second
    o, lse, status = bad_attention(change)
    assert status == lbx.LBX_ETREE and (o == 55.0).all() and (lse == 55.0).all()
    inp = commit_case([15, 31], [22, 22], [3, 20], 16)
    change(inp)
    k, v, out, status = run_commit(inp)
    assert status == lbx.LBX_ETREE and out == [-3, -3]
    assert same_bits(k, inp["k_pages"]) and same_bits(v, inp["v_pages"])


def test_a_tree_of_65_nodes_is_refused():
    inp = R.make_attention([4], [65], 1, 1, 64, 16, kind="chain", seed=9)
    o, lse, status = run_attention(inp)
    assert status == lbx.LBX_ETREE and (o == 55.0).all()


@pytest.mark.parametrize("page_id", [-1, 10 ** 6, 2 ** 31 - 1])
def test_a_page_outside_the_pool_is_not_read(page_id):
    """It is reported, and the other requests' outputs are what they were."""
    inp = R.make_attention([40, 7, 500], [9, 30, 1], 4, 2, 128, 16, seed=9)
    clean, clean_lse, _ = run_attention(inp)
    inp["block_table"][1, 1] = page_id
    o, lse, status = run_attention(inp)
    assert status == lbx.LBX_EINVAL
    rest = list(range(9)) + [39]
    assert torch.equal(o[:, rest], clean[:, rest]) and torch.equal(lse[:, rest], clean_lse[:, rest])


# ---- commit --------------------------------------------------------------------

def commit_case(ctx, new, ends, page, Hkv=2, dh=64, L=2, dtype="bf16", kind="random", seed=0):
    inp = R.make_attention(ctx, new, Hkv, Hkv, dh, page, L=L, dtype=dtype, kind=kind, seed=seed)
    inp["accepted"] = torch.tensor([n - 1 if e == "last" else e for n, e in zip(new, ends)], dtype=torch.int32)
    return inp


def run_commit(inp, stream=None):
    d = {k: None if v is None else v.cuda() for k, v in inp.items()}
    out, status = i32([-3] * len(inp["ctx_len"])), status_word()
    torch.cuda.synchronize()
    lbx.lbx_page_commit(page_cfg(inp), d["start"], d["ctx_len"], d["block_table"], d["parent"],
                        d["accepted"], d["k_pages"], d["v_pages"], out, d_status=status, stream=stream)
    torch.cuda.synchronize()
    return d["k_pages"].cpu(), d["v_pages"].cpu(), out.cpu().tolist(), int(status.item())


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


COMMIT = {
    "root_only": dict(ctx=[5], new=[4], ends=[0], page=16),
    "over_a_page": dict(ctx=[15, 31], new=[22, 22], ends=["last", 20], page=16, seed=3),
    "chain": dict(ctx=[9], new=[64], ends=["last"], page=16, kind="chain"),
    "half_a_chain": dict(ctx=[9, 0], new=[64, 40], ends=[30, 5], page=32, kind="chain"),
    "star": dict(ctx=[60, 0], new=[64, 64], ends=["last", 1], page=64, kind="star", dtype="f16"),
    "ragged": dict(ctx=[7, 0, 90, 33], new=[9, 0, 64, 1], ends=["last", 77, 63, 0], page=16, seed=8),
    "wide": dict(ctx=[100] * 20, new=[22] * 20, ends=["last"] * 20, page=64, Hkv=4, dh=256, L=1),
}


@pytest.mark.parametrize("name", sorted(COMMIT))
def test_commit(name):
    inp = commit_case(**COMMIT[name])
    k, v, out, status = run_commit(inp)
    assert status == 0
    page, table, start = inp["k_pages"].shape[2], inp["block_table"].numpy(), inp["start"].tolist()
    kr, vr = inp["k_pages"].clone(), inp["v_pages"].clone()
    for b, t in enumerate(inp["ctx_len"].tolist()):
        s, n = start[b], start[b + 1] - start[b]
        path = R.root_path(inp["parent"][s:s + n].tolist(), int(inp["accepted"][b])) if n else []
        for i, m in enumerate(path):
            (to, at), (frm, off) = (R.place(table, b, t + j, page) for j in (i, m))
            kr[:, to, at], vr[:, to, at] = kr[:, frm, off].clone(), vr[:, frm, off].clone()
        assert out[b] == t + len(path)
    assert same_bits(k, kr) and same_bits(v, vr)


@pytest.mark.parametrize("b,value", [(0, -1), (1, 22), (0, 2 ** 31 - 1)])
def test_bad_commits_move_nothing(b, value):
    inp = commit_case([15, 31], [22, 22], [3, 20], 16)
    inp["accepted"][b] = value
    k, v, out, status = run_commit(inp)
    assert status == lbx.LBX_ETREE and out == [-3, -3]
    assert same_bits(k, inp["k_pages"]) and same_bits(v, inp["v_pages"])


def test_a_path_through_a_page_outside_the_pool_does_not_move():
    inp = commit_case([15, 31], [22, 22], ["last", "last"], 16, kind="chain")
    inp["parent"][22:] = torch.tensor([-1] + [0] * 21)  # request 1: node 21 comes to place 1
    good = run_commit(inp)
    inp["block_table"][0, 1] = 999
    k, v, out, status = run_commit(inp)
    assert status == lbx.LBX_EINVAL and out == good[2]
    assert same_bits(k, good[0]) and same_bits(v, good[1])  # (a chain's path stays where it is)


# ---- together -------------------------------------------------------------------

def serve(steps=3, graph=False):
    """Prompts in, then rounds of a draft tree, its attention and its commit, with pages
    taken and given back; the same queries over contiguous keys for comparison."""
    Hq, Hkv, dh, page, B, L = 6, 2, 128, 16, 3, 2
    g = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(3)
    n_pages, width = 64, 20
    dev = dict(device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, **dev)
    stack = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    held, held2, n_free, n_free2 = i32([0] * B), i32([0] * B), i32([n_pages]), i32([0])
    kp, vp = (torch.full((L, n_pages, page, Hkv, dh), float("nan"), dtype=torch.bfloat16, **dev) for _ in "kv")
    ctx, status = i32([0] * B), status_word()
    inv_freq = (1e4 ** (-torch.arange(32).double() / 32)).float().cuda()
    rc = lbx.make_rope_cfg([32])
    kept = [[] for _ in range(B)]  # (k, v) of each position, [L][Hkv][dh]
    for step in range(steps):
        new = [37, 16, 60] if step == 0 else [9, 22, 5]
        M = sum(new) + 3
        cfg = lbx.make_page_cfg(L, B, M, Hq, Hkv, dh, page, n_pages, width)
        start, slot, pos = i32([0] * (B + 1)), i32([0] * M), i32([0] * M)
        lbx.lbx_page_tables(cfg, ctx, i32(new), held, n_free, table, stack, held2, n_free2, start, slot,
                            pos, d_status=status)
        held, held2, n_free, n_free2 = held2, held, n_free2, n_free
        parent = None
        if step:
            trees = [R.tree(rng, n) for n in new]
            parent = i32([p for t in trees for p in t] + [-1] * 3)
            depth = [len(R.root_path(t, i)) - 1 for t in trees for i in range(len(t))]
            at = torch.repeat_interleave(ctx.cpu(), torch.tensor(new)) + torch.tensor(depth)
            pos[:sum(new)] = at.to(torch.int32).cuda()
        qkv = torch.randn(L, M, Hq + 2 * Hkv, dh, generator=g).to(torch.bfloat16).cuda()
        w = torch.ones(L, dh, **dev)
        q = torch.zeros(L, M, Hq, dh, dtype=torch.bfloat16, **dev)
        lbx.lbx_qk_norm_rope(cfg, rc, qkv, inv_freq, pos.view(1, M), slot, q, kp, vp, q_weight=w,
                             k_weight=w, d_status=status)
        o, lse = torch.zeros_like(q), torch.zeros(L, M, Hq, **dev)
        lbx.lbx_paged_attention(cfg, start, ctx, table, q, kp, vp, o, lbx.new_paged_workspace(cfg),
                                parent=parent, lse=lse, d_status=status)
        inp = {"start": start.cpu(), "ctx_len": ctx.cpu(), "block_table": table.cpu(),
               "parent": None if parent is None else parent.cpu(), "q": q.cpu(), "k_pages": kp.cpu(),
               "v_pages": vp.cpu()}
        ref, ref_lse, tol, lse_tol = R.attention(inp)
        live = sum(new)
        assert (np.abs(o.cpu().double().numpy() - ref)[:, :live] <= tol[:, :live]).all()
        assert (np.abs(lse.cpu().double().numpy() - ref_lse)[:, :live] <= lse_tol[:, :live]).all()
        # the keys of positions kept so far are where the tables say
        for b, pairs in enumerate(kept):
            for p, (k1, v1) in enumerate(pairs):
                pg, off = R.place(inp["block_table"], b, p, page)
                assert torch.equal(inp["k_pages"][:, pg, off], k1) and torch.equal(inp["v_pages"][:, pg, off], v1)
        ends = [n - 1 for n in new]
        for b in range(B):
            t, s = int(ctx[b]), sum(new[:b])
            path = R.root_path(trees[b], ends[b]) if step else range(new[b])
            for m in path:
                pg, off = R.place(inp["block_table"], b, t + m, page)
                kept[b].append((inp["k_pages"][:, pg, off].clone(), inp["v_pages"][:, pg, off].clone()))
        if step:
            out = i32([0] * B)
            lbx.lbx_page_commit(cfg, start, ctx, table, parent, i32(ends), kp, vp, out, d_status=status)
            ctx = out
        else:
            ctx = i32([t + n for t, n in zip(ctx.tolist(), new)])
        assert ctx.tolist() == [len(p) for p in kept]
        assert int(n_free) + int(held.sum()) == n_pages
    # all requests end: every page comes back
    cfg = lbx.make_page_cfg(1, B, 1, 1, 1, 64, page, n_pages, width)
    lbx.lbx_page_tables(cfg, i32([0] * B), i32([0] * B), held, n_free, table, stack, held2, n_free2,
                        i32([0] * (B + 1)), i32([0]), i32([0]), d_status=status)
    assert int(n_free2) == n_pages and sorted(stack.tolist()) == list(range(n_pages))
    assert int(status.item()) == 0


def test_a_server_of_prompts_and_trees():
    serve(steps=6)


def test_the_example_serves():
    """Pages add up, paths are accepted, and the last round's attention is the definition's."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import paged_cache
    s, out = paged_cache.main(["--rounds", "4", "--chunk", "70"])
    ctx, held = s.ctx.tolist(), s.held.tolist()
    assert int(s.n_free) + sum(held) == paged_cache.N_PAGES
    assert all(c >= p + 4 for c, p in zip(ctx, paged_cache.PROMPTS)) and sum(ctx) > sum(paged_cache.PROMPTS) + 12
    inp = {k: out[k].cpu() for k in ("start", "ctx_len", "block_table", "parent", "q", "k_pages", "v_pages")}
    ref, ref_lse, tol, lse_tol = R.attention(inp)
    live = int(inp["start"][-1])
    assert (np.abs(out["o"].cpu().double().numpy() - ref)[:, :live] <= tol[:, :live]).all()
    assert (np.abs(out["lse"].cpu().double().numpy() - ref_lse)[:, :live] <= lse_tol[:, :live]).all()


@pytest.mark.parametrize("kind", ["decode", "chunk", "tree"])
def test_a_step_in_a_graph(kind):
    """All four calls captured once and replayed with other lengths, tokens and trees in the
    same arrays: each replay is what the calls give then."""
    B, page, Hq, Hkv, dh, L, M, width, n_pages = 3, 16, 8, 2, 128, 2, 150, 40, 130
    cfg = lbx.make_page_cfg(L, B, M, Hq, Hkv, dh, page, n_pages, width)
    rc, g = lbx.make_rope_cfg([24]), torch.Generator().manual_seed(4)
    a = {k: i32(np.zeros(n)) for k, n in (("ctx_len", B), ("new_len", B), ("held", B), ("n_free", 1),
                                          ("held_out", B), ("n_free_out", 1), ("start", B + 1), ("slot", M),
                                          ("pos", M), ("accepted", B), ("ctx_out", B), ("parent", M))}
    a["block_table"], a["free_list"] = i32(np.zeros((B, width))), i32(np.arange(n_pages))
    a["inv_freq"] = (1e4 ** (-torch.arange(24).double() / 24)).float().cuda()
    a["qkv"] = torch.zeros(L, M, Hq + 2 * Hkv, dh, dtype=torch.bfloat16, device="cuda")
    for k, shape in (("k_pages", (L, n_pages, page, Hkv, dh)), ("v_pages", (L, n_pages, page, Hkv, dh)),
                     ("q", (L, M, Hq, dh)), ("o", (L, M, Hq, dh))):
        a[k] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    a["lse"], status, ws = torch.zeros(L, M, Hq, device="cuda"), status_word(), lbx.new_paged_workspace(cfg)

    def calls():
        lbx.lbx_page_tables(cfg, a["ctx_len"], a["new_len"], a["held"], a["n_free"], a["block_table"],
                            a["free_list"], a["held_out"], a["n_free_out"], a["start"], a["slot"], a["pos"],
                            d_status=status)
        lbx.lbx_qk_norm_rope(cfg, rc, a["qkv"], a["inv_freq"], a["pos"].view(1, M), a["slot"], a["q"],
                             a["k_pages"], a["v_pages"], d_status=status)
        lbx.lbx_paged_attention(cfg, a["start"], a["ctx_len"], a["block_table"], a["q"], a["k_pages"],
                                a["v_pages"], a["o"], ws, parent=a["parent"] if kind == "tree" else None,
                                lse=a["lse"], d_status=status)
        if kind == "tree":
            lbx.lbx_page_commit(cfg, a["start"], a["ctx_len"], a["block_table"], a["parent"], a["accepted"],
                                a["k_pages"], a["v_pages"], a["ctx_out"], d_status=status)

    def fill(seed):
        rng = np.random.default_rng(seed)
        ctx = rng.integers(0, 400, B)
        new = np.ones(B, int) if kind == "decode" else rng.integers(1, 40 if kind == "tree" else 50, B)
        a["ctx_len"].copy_(i32(ctx)), a["new_len"].copy_(i32(new)), a["held"].zero_()
        a["n_free"].fill_(n_pages), a["free_list"].copy_(i32(rng.permutation(n_pages)))
        a["qkv"].copy_((torch.randn(a["qkv"].shape, generator=g) * 2).to(torch.bfloat16))
        for k in ("k_pages", "v_pages"):
            a[k].copy_(torch.randn(a[k].shape, generator=g).to(torch.bfloat16))
        trees = [p for n in new for p in R.tree(rng, int(n))]
        a["parent"][:len(trees)] = i32(trees)
        a["accepted"].copy_(i32(new - 1))

    side = torch.cuda.Stream()
    fill(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    outs = ("held_out", "n_free_out", "start", "slot", "pos", "block_table", "free_list", "q", "k_pages",
            "v_pages", "o", "lse", "ctx_out")
    for seed in (1, 2, 3):
        fill(seed)
        start = {k: v.clone() for k, v in a.items()}
        graph.replay()
        torch.cuda.synchronize()
        got = {k: a[k].clone() for k in outs}
        for k, v in start.items():
            a[k].copy_(v)
        calls()
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(got[k].view(torch.uint8) if got[k].is_floating_point() else got[k],
                               a[k].view(torch.uint8) if got[k].is_floating_point() else a[k]), (seed, k)
    assert int(status.item()) == 0


def test_calls_side_by_side_and_on_one_workspace():
    """Calls of all head dimensions and lengths take turns on one workspace, and run on two
    streams with a workspace each: the bits are those of calls by themselves."""
    cases = [R.make_attention([900, 30], [1, 1], 8, 2, 64, 16, seed=1),
             R.make_attention([3000, 700, 5], [40, 300, 1], 8, 2, 128, 32, seed=2),
             R.make_attention([2500], [22], 12, 2, 256, 64, kind="random", seed=3),
             R.make_attention([0], [1500], 8, 1, 128, 64, dtype="f16", seed=4),
             R.make_attention([5000, 1], [1, 1], 8, 2, 256, 16, seed=5)]
    alone = [run_attention(c) for c in cases]
    cfgs = [page_cfg(c) for c in cases]
    size = max(lbx.lbx_paged_workspace_size(c) for c in cfgs)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    dev = [{k: None if v is None else v.cuda() for k, v in c.items()} for c in cases]
    outs = [[(torch.zeros_like(d["q"]), torch.zeros(d["q"].shape[:-1], device="cuda")) for d in dev]
            for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s in range(2):
            for i in range(len(cases)) if s == 0 else reversed(range(len(cases))):
                d, (o, lse) = dev[i], outs[s][i]
                lbx.lbx_paged_attention(cfgs[i], d["start"], d["ctx_len"], d["block_table"], d["q"],
                                        d["k_pages"], d["v_pages"], o, spaces[s], parent=d["parent"], lse=lse,
                                        stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for (o, lse), (ref_o, ref_lse, _) in zip(outs[s], alone):
            assert torch.equal(o.cpu(), ref_o)
            assert torch.equal(lse.cpu(), ref_lse)


@pytest.mark.parametrize("dh,dtype", [(64, "bf16"), (128, "f16"), (256, "bf16")])
def test_single_tokens_with_scores_of_minus_infinity_and_nan(dh, dtype):
    """As above for the few rows of a decode step, over one unit of keys and over many."""
    inp = R.make_attention([20, 1000, 300, 900], [1, 1, 1, 1], 4, 2, dh, 16, dtype=dtype, seed=6)
    clean, clean_lse, _ = run_attention(inp)
    q, k = inp["q"], inp["k_pages"]
    q[:, [0, 3]] = q[:, [0, 3]].abs() + 0.5
    for b, n in ((0, 21), (3, 901)):
        for p in range(n):
            k[:, inp["block_table"][b, p // 16], p % 16] = -torch.inf
    q[0, 1, 2, 5] = torch.nan
    o, lse, status = run_attention(inp)
    assert status == 0
    assert (o[:, [0, 3]] == 0).all() and (lse[:, [0, 3]] == -torch.inf).all()
    assert o[0, 1, 2].isnan().all() and lse[0, 1, 2].isnan()
    assert torch.equal(o[:, 2], clean[:, 2]) and torch.equal(lse[:, 2], clean_lse[:, 2])
    assert torch.equal(o[0, 1, [0, 1, 3]], clean[0, 1, [0, 1, 3]])


FEW = {
    "unit_edges": dict(ctx=[126, 127, 128, 255, 256], new=[1] * 5, Hq=4, Hkv=2, dh=128, page=16),
    "rows_8": dict(ctx=[500, 3], new=[2, 1], Hq=8, Hkv=2, dh=64, page=32, dtype="f16"),
    "chunk_of_8": dict(ctx=[300, 0], new=[8, 5], Hq=3, Hkv=3, dh=256, page=64),
    "tree_of_8": dict(ctx=[300, 0, 127], new=[8, 1, 6], Hq=3, Hkv=3, dh=128, page=16, kind="random"),
    "tree_over_a_unit": dict(ctx=[125], new=[7], Hq=1, Hkv=1, dh=64, page=256, kind="star", dtype="f16"),
    "many_units": dict(ctx=[9000], new=[1], Hq=6, Hkv=1, dh=256, page=64),
    "requests_100": dict(ctx=[(7 * b) % 120 for b in range(100)], new=[b % 2 for b in range(100)], Hq=4, Hkv=1,
                         dh=128, page=16),
    "requests_60_layers": dict(ctx=[(7 * b) % 90 for b in range(60)], new=[1] * 60, Hq=8, Hkv=2, dh=64, page=32,
                               L=2, pad=3),
    "rows_9_beside_1": dict(ctx=[40, 700], new=[9, 1], Hq=2, Hkv=2, dh=128, page=16),
}


@pytest.mark.parametrize("name", sorted(FEW))
def test_few_rows(name):
    check_attention(R.make_attention(**FEW[name], seed=900 + len(name)), calls=2)
