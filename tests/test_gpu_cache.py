"""GPU parity of the bounded, shared cache's operators with their definitions in
64 bits, through the C ABI.  The error bounds are derived in cache_ref; whole
numbers, moved rows and everything that must stay untouched compare equal."""
import numpy as np
import pytest
import torch

import cache_ref as R
from tree_verify_linear_gb300 import lbx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for -m gpu tests")
    from tree_verify_linear_gb300 import build
    build.build()
    lbx.load()


def cfg_of(inp, **kw):
    L, Bq, N, Hq, dh = inp["q"].shape
    P = inp["k_prefix"].shape[1] if "k_prefix" in inp else 0
    return lbx.make_attn_cfg(
        L=L, Bq=Bq, N=N, Hq=Hq, Hkv=inp["k_tree"].shape[3], dh=dh, T=inp["k_cache"].shape[2], P=P,
        dtype=lbx.LBX_F16 if inp["q"].dtype == torch.float16 else lbx.LBX_BF16, **kw)


def run_attention(inp, calls=1, want_lse=True, stream=None, **kw):
    cfg = cfg_of(inp, **kw)
    d = {k: v.cuda() for k, v in inp.items()}
    o = torch.full_like(d["q"], float("nan"))
    lse = torch.full(o.shape[:-1], float("nan"), device="cuda") if want_lse else None
    ws, status = lbx.new_cache_attn_workspace(cfg), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pre = (d["k_prefix"], d["v_prefix"]) if cfg.P else ()
    call = lbx.lbx_prefix_attention if cfg.P else lbx.lbx_window_attention
    for _ in range(calls):
        call(cfg, d["ctx_len"], d["parent"], d["q"], *pre, d["k_cache"], d["v_cache"], d["k_tree"],
             d["v_tree"], o, ws, lse=lse, d_status=status, stream=stream)
    torch.cuda.synchronize()
    return o.cpu(), None if lse is None else lse.cpu(), int(status.item())


def check_attention(inp, **kw):
    o, lse, status = run_attention(inp, **kw)
    assert status == 0
    ref_o, ref_lse, o_tol, lse_tol = R.attention(inp, prefix="k_prefix" in inp, **kw)
    over = np.abs(o.double().numpy() - ref_o) / o_tol
    assert np.isfinite(over).all() and over.max() <= 1, float(over.max())
    over = np.abs(lse.double().numpy() - ref_lse) / lse_tol
    assert np.isfinite(over).all() and over.max() <= 1, float(over.max())
    return o, lse


# name: (sizes, window, n_sink)
ATTN = {
    "one_token": (dict(L=1, Bq=1, N=1, Hq=1, Hkv=1, dh=64, T=1), 0, 0),
    "one_token_no_cache": (dict(L=1, Bq=2, N=1, Hq=2, Hkv=1, dh=128, T=0), 0, 0),
    "empty_contexts": (dict(L=1, Bq=2, N=3, Hq=2, Hkv=2, dh=256, T=70, ctx=[0, 0]), 5, 1),
    "window_one": (dict(L=1, Bq=2, N=9, Hq=4, Hkv=2, dh=64, T=40), 1, 0),
    "window_one_sinks": (dict(L=1, Bq=2, N=9, Hq=4, Hkv=2, dh=64, T=40), 1, 5),
    "window_inside_the_tree": (dict(L=1, Bq=2, N=40, Hq=2, Hkv=1, dh=128, T=30, tree="chain"), 9, 2),
    "window_64": (dict(L=2, Bq=2, N=22, Hq=12, Hkv=2, dh=256, T=300, ctx=[300, 129]), 64, 4),
    "window_63_sinks_past_start": (dict(L=1, Bq=3, N=7, Hq=6, Hkv=2, dh=128, T=200, dtype="f16",
                                        ctx=[200, 63, 64]), 63, 150),
    "window_longer_than_context": (dict(L=1, Bq=2, N=5, Hq=4, Hkv=4, dh=64, T=90), 1000, 4),
    "sinks_65": (dict(L=1, Bq=1, N=4, Hq=4, Hkv=1, dh=128, T=500, ctx=[470]), 100, 65),
    "sinks_128": (dict(L=1, Bq=1, N=4, Hq=4, Hkv=1, dh=64, T=500, ctx=[500]), 128, 128),
    "rows_129": (dict(L=1, Bq=1, N=43, Hq=3, Hkv=1, dh=256, T=140, ctx=[131]), 0, 0),
    "rows_132": (dict(L=2, Bq=2, N=22, Hq=24, Hkv=4, dh=256, T=150), 0, 0),
    "rows_384": (dict(L=1, Bq=1, N=64, Hq=6, Hkv=1, dh=128, T=260, ctx=[257]), 100, 3),
    "rows_512_f16": (dict(L=1, Bq=1, N=64, Hq=8, Hkv=1, dh=64, T=130, dtype="f16", ctx=[127]), 0, 0),
    "chain_64": (dict(L=1, Bq=2, N=64, Hq=2, Hkv=2, dh=64, T=100, tree="chain"), 30, 2),
    "star_64": (dict(L=1, Bq=2, N=64, Hq=2, Hkv=1, dh=256, T=64, tree="star", ctx=[64, 1]), 0, 0),
    "group_of_48": (dict(L=1, Bq=1, N=3, Hq=48, Hkv=1, dh=64, T=77), 0, 0),
    "group_of_130": (dict(L=1, Bq=1, N=2, Hq=130, Hkv=1, dh=128, T=90, ctx=[81]), 0, 0),
    "group_of_65": (dict(L=1, Bq=2, N=3, Hq=130, Hkv=2, dh=256, T=70, dtype="f16"), 40, 2),
    "many_heads": (dict(L=1, Bq=2, N=1, Hq=64, Hkv=64, dh=64, T=50), 20, 1),
    "ragged_f16": (dict(L=2, Bq=5, N=4, Hq=8, Hkv=2, dh=128, T=333, dtype="f16",
                        ctx=[333, 0, 1, 64, 128]), 0, 0),
    "wide_scores": (dict(L=1, Bq=2, N=6, Hq=4, Hkv=2, dh=256, T=400, ctx=[400, 300], width=20.0), 0, 0),
    "long": (dict(L=1, Bq=1, N=2, Hq=2, Hkv=1, dh=128, T=5000, ctx=[4999]), 0, 0),
    "long_f16": (dict(L=1, Bq=1, N=2, Hq=2, Hkv=1, dh=256, T=5000, dtype="f16", ctx=[5000]), 4097, 7),
}


@pytest.mark.parametrize("name", sorted(ATTN))
def test_window_attention(name):
    sizes, window, n_sink = ATTN[name]
    check_attention(R.make_inputs(**sizes, seed=100 + len(name)), window=window, n_sink=n_sink)


PREFIX = {
    "one_key": dict(L=1, Bq=1, N=1, Hq=1, Hkv=1, dh=64, T=0, P=1),
    "one_request": dict(L=1, Bq=1, N=5, Hq=6, Hkv=2, dh=256, T=70, P=64),
    "odd": dict(L=2, Bq=3, N=7, Hq=6, Hkv=2, dh=128, T=90, P=201, ctx=[90, 0, 33]),
    "rows_660": dict(L=1, Bq=5, N=22, Hq=6, Hkv=1, dh=256, T=130, P=129),
    "rows_129": dict(L=1, Bq=43, N=1, Hq=3, Hkv=1, dh=64, T=9, P=300, dtype="f16"),
    "wide_batch": dict(L=1, Bq=70, N=2, Hq=16, Hkv=2, dh=64, T=5, P=65, dtype="f16"),
    "no_cache": dict(L=2, Bq=4, N=3, Hq=4, Hkv=4, dh=128, T=0, P=127),
    "long": dict(L=1, Bq=2, N=1, Hq=4, Hkv=2, dh=128, T=100, P=4097),
    "long_256": dict(L=1, Bq=3, N=2, Hq=6, Hkv=1, dh=256, T=10, P=3000, dtype="f16", ctx=[10, 0, 5]),
}


@pytest.mark.parametrize("name", sorted(PREFIX))
def test_prefix_attention(name):
    check_attention(R.make_inputs(**PREFIX[name], seed=200 + len(name)))


# Enough keys that every CTA walks many blocks and several streams, whole ones
# among them, with lengths that differ from request to request.
BUSY = {
    "dh256_two_tiles": (dict(L=4, Bq=4, N=22, Hq=12, Hkv=2, dh=256, T=3000, ctx=[3000, 1, 1501, 2111]), 0, 0),
    "dh256_window": (dict(L=8, Bq=3, N=9, Hq=8, Hkv=4, dh=256, T=2500, ctx=[2500, 700, 2047]), 1100, 70),
    "dh128_one_row": (dict(L=4, Bq=6, N=1, Hq=8, Hkv=8, dh=128, T=4000,
                           ctx=[4000, 3999, 0, 2222, 127, 3100]), 0, 0),
    "dh128_f16": (dict(L=4, Bq=6, N=5, Hq=32, Hkv=8, dh=128, T=2100, dtype="f16",
                       ctx=[2100, 2000, 1999, 64, 129, 1024]), 0, 0),
    "dh64_three_tiles": (dict(L=3, Bq=4, N=64, Hq=30, Hkv=5, dh=64, T=2000, ctx=[2000, 77, 1231, 640]), 0, 0),
    "dh64_f16_window": (dict(L=9, Bq=5, N=3, Hq=16, Hkv=8, dh=64, T=3000, dtype="f16",
                             ctx=[3000, 2900, 511, 1025, 2001]), 1500, 3),
    # one or two streams over the whole GPU: joins of many pieces
    "one_stream_pair": (dict(L=1, Bq=1, N=22, Hq=6, Hkv=1, dh=256, T=9000, ctx=[8990]), 0, 0),
    "one_stream_few_rows": (dict(L=1, Bq=1, N=3, Hq=6, Hkv=1, dh=256, T=9000, dtype="f16", ctx=[9000]), 0, 0),
    "two_streams_dh128": (dict(L=1, Bq=2, N=40, Hq=7, Hkv=1, dh=128, T=7000, ctx=[7000, 5001]), 0, 0),
    "one_stream_dh64": (dict(L=1, Bq=1, N=12, Hq=4, Hkv=1, dh=64, T=20000, ctx=[19999]), 0, 0),
    "one_prefix": (dict(L=1, Bq=7, N=22, Hq=5, Hkv=1, dh=128, T=60, P=9001, dtype="f16"), 0, 0),
    "prefix_dh256": (dict(L=3, Bq=5, N=22, Hq=12, Hkv=2, dh=256, T=700, P=3001, ctx=[700, 3, 501, 258, 640]), 0, 0),
    "prefix_dh128_f16": (dict(L=3, Bq=9, N=7, Hq=32, Hkv=4, dh=128, T=900, P=4000, dtype="f16"), 0, 0),
    "prefix_dh64": (dict(L=4, Bq=40, N=2, Hq=16, Hkv=4, dh=64, T=300, P=2049), 0, 0),
}


@pytest.mark.parametrize("name", sorted(BUSY))
def test_long_ragged_batches(name):
    sizes, window, n_sink = BUSY[name]
    inp = R.make_inputs(**sizes, seed=500 + len(name))
    o, lse, status = run_attention(inp, window=window, n_sink=n_sink)
    assert status == 0
    ref_o, ref_lse, o_tol, lse_tol = R.attention_dense(inp, window=window, n_sink=n_sink)
    over = np.abs(o.double().numpy() - ref_o) / o_tol
    assert np.isfinite(over).all() and over.max() <= 1, float(over.max())
    over = np.abs(lse.double().numpy() - ref_lse) / lse_tol
    assert np.isfinite(over).all() and over.max() <= 1, float(over.max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.3, 1.0])
def test_other_scales(dtype, scale):
    check_attention(R.make_inputs(1, 2, 4, 4, 2, 64, 150, dtype=dtype, seed=7, width=0.5), scale=scale)


def test_lse_may_be_left_out():
    inp = R.make_inputs(1, 2, 6, 4, 2, 128, 90, seed=8)
    o, _, _ = run_attention(inp)
    o2, _, status = run_attention(inp, want_lse=False)
    assert status == 0 and torch.equal(o, o2)


@pytest.mark.parametrize("P,sizes", [
    (0, dict(L=2, Bq=3, N=22, Hq=12, Hkv=2, dh=256, T=400, ctx=[400, 20, 333])),
    (140, dict(L=2, Bq=3, N=22, Hq=12, Hkv=2, dh=256, T=400, ctx=[400, 20, 333])),
    (0, dict(L=1, Bq=2, N=22, Hq=6, Hkv=1, dh=128, T=9000, ctx=[9000, 8001])),
    (0, dict(L=3, Bq=5, N=9, Hq=8, Hkv=4, dh=256, T=3000, dtype="f16")),
    (5000, dict(L=1, Bq=6, N=5, Hq=8, Hkv=2, dh=64, T=700)),
])
def test_calls_in_a_row_and_on_another_stream_agree(P, sizes):
    inp = R.make_inputs(**sizes, P=P, seed=9)
    a, al, _ = run_attention(inp)
    b, bl, _ = run_attention(inp, calls=3)
    c, cl, status = run_attention(inp, calls=2, stream=torch.cuda.Stream())
    assert status == 0
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(al, bl) and torch.equal(al, cl)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dh,window,n_sink", [(64, 0, 0), (128, 40, 3), (256, 100, 70)])
def test_positions_no_query_sees_may_hold_anything(bad, dh, window, n_sink):
    inp = R.make_inputs(1, 4, 5, 4, 2, dh, 300, ctx=[300, 0, 201, 64], seed=10)
    o, lse, _ = run_attention(inp, window=window, n_sink=n_sink)
    dirty = {k: v.clone() for k, v in inp.items()}
    for b in range(4):
        ctx = int(inp["ctx_len"][b])
        first = max(0, ctx - window + 1) if window else 0
        for k in ("k_cache", "v_cache"):
            dirty[k][:, b, ctx:] = bad
            dirty[k][:, b, min(n_sink, first):first] = bad
    o2, lse2, status = run_attention(dirty, window=window, n_sink=n_sink)
    assert status == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_garbage_past_short_caches_beside_a_prefix():
    inp = R.make_inputs(1, 3, 4, 4, 2, 128, 100, P=77, ctx=[0, 65, 100], seed=11)
    o, lse, _ = run_attention(inp)
    for b in range(3):
        for k in ("k_cache", "v_cache"):
            inp[k][:, b, int(inp["ctx_len"][b]):] = float("nan")
    o2, lse2, status = run_attention(inp)
    assert status == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_a_query_without_a_finite_score(dh):
    """Its keys all score -inf: o = 0 and lse = -inf; the other request is as before."""
    inp = R.make_inputs(1, 2, 1, 2, 1, dh, 70, ctx=[3, 70], seed=12)
    inp["q"] = inp["q"].abs() + 1
    o, lse, _ = run_attention(inp)
    inp["k_cache"][:, 0, :3] = -float("inf")
    inp["k_tree"][:, 0] = -float("inf")
    o2, lse2, status = run_attention(inp)
    assert status == 0
    assert not o2[:, 0].any() and (lse2[:, 0] == -torch.inf).all()
    assert torch.equal(o[:, 1], o2[:, 1]) and torch.equal(lse[:, 1], lse2[:, 1])


def test_lowest_and_infinite_scores_among_finite_ones():
    """Keys that score the type's lowest value or -inf weigh nothing."""
    inp = R.make_inputs(1, 1, 3, 2, 1, 64, 200, ctx=[200], seed=13)
    inp["q"] = inp["q"].abs() + 0.5
    inp["k_cache"][:, :, 10:60] = -float("inf")
    inp["k_cache"][:, :, 60:140] = torch.finfo(torch.bfloat16).min
    o, lse, status = run_attention(inp)
    assert status == 0
    keep = torch.cat([torch.arange(10), torch.arange(140, 200)])
    small = dict(inp, k_cache=inp["k_cache"][:, :, keep], v_cache=inp["v_cache"][:, :, keep],
                 ctx_len=torch.tensor([70], dtype=torch.int32))
    ref_o, ref_lse, o_tol, lse_tol = R.attention(small)
    assert (np.abs(o.double().numpy() - ref_o) <= o_tol).all()
    assert (np.abs(lse.double().numpy() - ref_lse) <= lse_tol).all()


def test_offsets_past_32_bits():
    """The last request of a cache of more than 2^31 elements."""
    L, Bq, T, Hkv, dh = 1, 3, 900_000, 4, 256
    assert Bq * T * Hkv * dh > 1 << 31
    small = R.make_inputs(1, Bq, 2, 4, Hkv, dh, 100, ctx=[100] * 3, seed=14)
    cfg = lbx.make_attn_cfg(L, Bq, 2, 4, Hkv, dh, T, window=80, n_sink=5)
    d = {k: v.cuda() for k, v in small.items()}
    kc, vc = (torch.zeros(L, Bq, T, Hkv, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # the same 100 positions at the cache's end; the first five as sinks
    for big, k in ((kc, "k_cache"), (vc, "v_cache")):
        big[:, :, T - 100:] = d[k]
        big[:, :, :5] = d[k][:, :, :5]
    ctx = torch.full((Bq,), T, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(d["q"]), torch.empty(L, Bq, 2, 4, device="cuda")
    lbx.lbx_window_attention(cfg, ctx, d["parent"], d["q"], kc, vc, d["k_tree"], d["v_tree"], o,
                             lbx.new_cache_attn_workspace(cfg), lse=lse)
    ref_o, ref_lse, o_tol, lse_tol = R.attention(small, window=80, n_sink=5)
    assert (np.abs(o.cpu().double().numpy() - ref_o) <= o_tol).all()
    assert (np.abs(lse.cpu().double().numpy() - ref_lse) <= lse_tol).all()
    # weights and eviction over the same cache
    score = torch.zeros(L, Bq, Hkv, T, device="cuda")
    tree = torch.empty(L, Bq, Hkv, 2, device="cuda")
    lbx.lbx_attention_mass(cfg, ctx, d["parent"], d["accepted"], d["q"], lse, kc, d["k_tree"],
                           score, tree)
    at = torch.cat([torch.arange(5), torch.arange(T - 95, T)]).cuda()
    ref, ref_tree, tol, tree_tol = R.mass(small, lse.cpu().numpy(), np.zeros((L, Bq, Hkv, 100)),
                                          window=80, n_sink=5)
    assert (np.abs(score[..., at].cpu().numpy() - ref) <= tol).all()
    assert (np.abs(tree.cpu().numpy() - ref_tree) <= tree_tol).all()
    assert float(score.sum()) == pytest.approx(float(score[..., at].sum()), rel=1e-6)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(L, Bq, Hkv, T).contiguous()
    out = [torch.empty(Bq, dtype=torch.int32, device="cuda") for _ in range(2)]
    lbx.lbx_cache_evict(cfg, T // 2, 100, ctx, ctx, d["parent"], d["accepted"], d["k_tree"],
                        d["v_tree"], tree, kc, vc, score, pos, *out)
    assert out[0].tolist() == [T // 2] * 3
    path = [len(R.root_path(small["parent"][b].tolist(), int(small["accepted"][b]))) for b in range(3)]
    for b in range(Bq):
        # the recent entries were the only ones past the middle worth keeping,
        # and fill the highest-numbered free places in order
        new = pos[0, b, 0, :T // 2].cpu()
        moved = (new >= T // 2).nonzero()[:, 0]
        assert new[moved].tolist() == list(range(T + path[b] - 100, T + path[b]))
        held = small["k_cache"][0, b, path[b]:, 0]
        assert torch.equal(kc[0, b, moved[:100 - path[b]].cuda(), 0].cpu(), held)


# ---- weights per key ----------------------------------------------------------

def run_mass(inp, lse, score, **kw):
    cfg = cfg_of(inp, **kw)
    d = {k: v.cuda() for k, v in inp.items()}
    L, Bq, N, Hq, dh = inp["q"].shape
    s = torch.from_numpy(score).cuda()
    tree = torch.full((L, Bq, cfg.Hkv, N), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lbx.lbx_attention_mass(cfg, d["ctx_len"], d["parent"], d["accepted"], d["q"], lse.cuda(),
                           d["k_cache"], d["k_tree"], s, tree, status)
    torch.cuda.synchronize()
    return s.cpu().numpy(), tree.cpu().numpy(), int(status.item())


MASS = {k: ATTN[k] for k in ATTN if k not in ("many_heads", "wide_scores")}


@pytest.mark.parametrize("name", sorted(MASS))
def test_attention_mass(name):
    sizes, window, n_sink = MASS[name]
    inp = R.make_inputs(**sizes, seed=300 + len(name))
    _, ref_lse, _, _ = R.attention(inp, window=window, n_sink=n_sink)
    lse = torch.from_numpy(ref_lse.astype(np.float32))
    L, Bq, T, Hkv = inp["k_cache"].shape[:4]
    score = np.random.default_rng(1).random((L, Bq, Hkv, T)).astype(np.float32)
    got, tree, status = run_mass(inp, lse, score, window=window, n_sink=n_sink)
    ref, ref_tree, tol, tree_tol = R.mass(inp, lse.numpy(), score, window=window, n_sink=n_sink)
    assert status == 0
    assert (np.abs(got - ref) <= tol).all() and (np.abs(tree - ref_tree) <= tree_tol).all()
    for b in range(Bq):
        ctx = int(inp["ctx_len"][b])
        assert np.array_equal(got[:, b, :, ctx:], score[:, b, :, ctx:])


@pytest.mark.parametrize("sizes", [
    dict(L=4, Bq=4, N=22, Hq=12, Hkv=2, dh=256, T=3000, ctx=[3000, 1, 1501, 2111]),
    dict(L=6, Bq=5, N=64, Hq=32, Hkv=8, dh=128, T=1500, dtype="f16", tree="chain"),
    dict(L=9, Bq=6, N=5, Hq=16, Hkv=4, dh=64, T=2500),
    dict(L=1, Bq=1, N=40, Hq=8, Hkv=1, dh=256, T=20000, ctx=[19999], tree="chain"),
])
def test_mass_of_long_ragged_batches(sizes):
    """Every CTA walks many blocks and several streams; paths longer than a pass."""
    inp = R.make_inputs(**sizes, seed=31)
    if sizes.get("tree") == "chain":
        inp["accepted"][:] = sizes["N"] - 1
    _, ref_lse, _, _ = R.attention_dense(inp)
    lse = torch.from_numpy(ref_lse.astype(np.float32))
    L, Bq, T, Hkv = inp["k_cache"].shape[:4]
    score = np.random.default_rng(2).random((L, Bq, Hkv, T)).astype(np.float32)
    got, tree, status = run_mass(inp, lse, score)
    ref, ref_tree, tol, tree_tol = R.mass_dense(inp, lse.numpy(), score)
    assert status == 0
    assert (np.abs(got - ref) <= tol).all() and (np.abs(tree - ref_tree) <= tree_tol).all()
    again, tree2, _ = run_mass(inp, lse, score)
    assert np.array_equal(got, again) and np.array_equal(tree, tree2)


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_mass_of_a_long_path_and_unseen_garbage(dh):
    """64 nodes on the path (512 query rows); NaN where no query looks; a query
    with lse = -inf adds nothing."""
    inp = R.make_inputs(1, 2, 64, 8, 1, dh, 150, ctx=[130, 7], tree="chain", seed=20)
    inp["accepted"][:] = 63
    _, ref_lse, _, _ = R.attention(inp)
    ref_lse[0, 1, 5] = -np.inf
    lse = torch.from_numpy(ref_lse.astype(np.float32))
    score = np.zeros((1, 2, 1, 150), np.float32)
    ref, ref_tree, tol, tree_tol = R.mass(inp, lse.numpy(), score)
    for b, ctx in enumerate((130, 7)):
        inp["k_cache"][:, b, ctx:] = float("nan")
    got, tree, status = run_mass(inp, lse, score)
    assert status == 0
    assert (np.abs(got - ref) <= tol).all() and (np.abs(tree - ref_tree) <= tree_tol).all()


# ---- eviction -------------------------------------------------------------------

def run_evict(inp, score, tree, pos, seen, budget, n_sink, n_recent):
    cfg = cfg_of(inp, n_sink=n_sink)
    d = {k: v.cuda() for k, v in inp.items()}
    s, p = torch.from_numpy(score).cuda(), torch.from_numpy(pos).cuda()
    Bq = cfg.Bq
    out = [torch.full((Bq,), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lbx.lbx_cache_evict(cfg, budget, n_recent, d["ctx_len"],
                        torch.tensor(seen, dtype=torch.int32, device="cuda"), d["parent"],
                        d["accepted"], d["k_tree"], d["v_tree"], torch.from_numpy(tree).cuda(),
                        d["k_cache"], d["v_cache"], s, p, *out, d_status=status)
    torch.cuda.synchronize()
    return (d["k_cache"].cpu(), d["v_cache"].cpu(), s.cpu().numpy(), p.cpu().numpy(),
            out[0].cpu().numpy(), out[1].cpu().numpy()), int(status.item())


# name: (sizes, budget, n_sink, n_recent, kind of scores)
EVICT = {
    "room_left": (dict(L=2, Bq=2, N=9, Hq=2, Hkv=2, dh=64, T=60, ctx=[20, 0]), 50, 4, 8, "random"),
    "just_full": (dict(L=1, Bq=1, N=1, Hq=1, Hkv=1, dh=64, T=33, ctx=[32]), 33, 0, 0, "random"),
    "one_over": (dict(L=1, Bq=2, N=1, Hq=4, Hkv=2, dh=256, T=64, ctx=[64, 63]), 64, 4, 8, "random"),
    "budget_one": (dict(L=1, Bq=2, N=5, Hq=1, Hkv=1, dh=128, T=50, ctx=[50, 0]), 1, 0, 0, "random"),
    "budget_below_path": (dict(L=1, Bq=2, N=30, Hq=1, Hkv=1, dh=64, T=40, ctx=[3, 40], tree="chain"),
                          7, 0, 0, "random"),
    "half": (dict(L=2, Bq=3, N=22, Hq=4, Hkv=4, dh=256, T=700, ctx=[700, 350, 349]), 350, 4, 64, "random"),
    "ties": (dict(L=1, Bq=2, N=8, Hq=2, Hkv=2, dh=64, T=500, ctx=[500, 77]), 100, 0, 0, "ties"),
    "all_equal": (dict(L=1, Bq=1, N=8, Hq=1, Hkv=1, dh=64, T=300, ctx=[300]), 130, 3, 5, "equal"),
    "special_scores": (dict(L=1, Bq=2, N=8, Hq=2, Hkv=2, dh=128, T=300, ctx=[300, 200]), 90, 0, 0, "special"),
    "all_protected": (dict(L=1, Bq=1, N=4, Hq=1, Hkv=1, dh=64, T=200, ctx=[200]), 60, 0, 1000, "random"),
    "sinks_only": (dict(L=1, Bq=1, N=4, Hq=1, Hkv=1, dh=64, T=200, ctx=[200]), 60, 50, 0, "random"),
    "f16": (dict(L=1, Bq=2, N=6, Hq=4, Hkv=2, dh=128, T=1100, dtype="f16", ctx=[1100, 1000]), 513, 4, 32, "random"),
    "long_moves": (dict(L=1, Bq=1, N=3, Hq=1, Hkv=1, dh=64, T=9000, ctx=[9000]), 4000, 4, 64, "late"),
    "keys_past_shared_memory": (dict(L=1, Bq=1, N=2, Hq=1, Hkv=1, dh=64, T=60000, ctx=[59999]), 30001, 9, 100, "ties"),
}


@pytest.mark.parametrize("name", sorted(EVICT))
def test_cache_evict(name):
    sizes, budget, n_sink, n_recent, kind = EVICT[name]
    inp = R.make_inputs(**sizes, seed=400 + len(name))
    L, Bq, T, Hkv = inp["k_cache"].shape[:4]
    N = inp["q"].shape[2]
    rng = np.random.default_rng(len(name))
    score = rng.lognormal(0, 2, (L, Bq, Hkv, T)).astype(np.float32)
    tree = rng.lognormal(0, 2, (L, Bq, Hkv, N)).astype(np.float32)
    if kind == "ties":
        score, tree = np.round(score).clip(0, 5), np.round(tree).clip(0, 5)
    if kind == "equal":
        score[:], tree[:] = 0.25, 0.25
    if kind == "late":
        score += np.arange(T, dtype=np.float32)
    if kind == "special":
        values = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.0, 1e-42, 3e38], np.float32)
        score = values[rng.integers(0, 8, score.shape)]
        tree = values[rng.integers(0, 8, tree.shape)]
    pos = np.stack([rng.permutation(2 * T)[:T] for _ in range(L * Bq * Hkv)]).astype(np.int32)
    pos = pos.reshape(L, Bq, Hkv, T)
    seen = [2 * T] * Bq
    got, status = run_evict(inp, score, tree, pos, seen, budget, n_sink, n_recent)
    assert status == 0
    ref = R.evict(inp, score, tree, pos, seen, budget, n_sink, n_recent)
    for name, a, b in zip(("k_cache", "v_cache", "score", "pos", "ctx_out", "seen_out"), got, ref):
        if isinstance(a, torch.Tensor):
            assert torch.equal(a, b), name
        else:
            assert a.tobytes() == b.tobytes(), name


def test_rounds_of_a_full_cache_keep_it_consistent():
    """Attention, weights and eviction in turn: after every round each cache
    holds `budget` distinct positions, the sinks and the recent ones among
    them, and pos says which key sits where."""
    L, Bq, N, Hq, Hkv, dh, budget = 2, 2, 6, 4, 2, 64, 48
    g = torch.Generator().manual_seed(3)
    every_k = torch.randn(L, Bq, 400, Hkv, dh, generator=g).bfloat16()
    inp = R.make_inputs(L, Bq, N, Hq, Hkv, dh, budget, ctx=[40, 48], tree="chain", seed=21)
    d = {k: v.cuda() for k, v in inp.items()}
    d["k_cache"][:] = every_k[:, :, :budget]
    cfg = cfg_of(inp, n_sink=2)
    score = torch.zeros(L, Bq, Hkv, budget, device="cuda")
    pos = torch.arange(budget, dtype=torch.int32, device="cuda").expand(L, Bq, Hkv, budget).contiguous()
    tree, o = torch.empty(L, Bq, Hkv, N, device="cuda"), torch.empty_like(d["q"])
    lse, ws = torch.empty(L, Bq, N, Hq, device="cuda"), lbx.new_cache_attn_workspace(cfg)
    ctx, seen = d["ctx_len"], d["ctx_len"].clone()
    for r in range(12):
        for b in range(Bq):
            d["k_tree"][:, b] = every_k[:, b, int(seen[b]):int(seen[b]) + N].cuda()
        acc = torch.tensor([r % N, (r * 5) % N], dtype=torch.int32, device="cuda")
        lbx.lbx_window_attention(cfg, ctx, d["parent"], d["q"], d["k_cache"], d["v_cache"], d["k_tree"],
                                 d["v_tree"], o, ws, lse=lse)
        lbx.lbx_attention_mass(cfg, ctx, d["parent"], acc, d["q"], lse, d["k_cache"], d["k_tree"], score, tree)
        ctx2, seen2 = torch.empty_like(ctx), torch.empty_like(ctx)
        lbx.lbx_cache_evict(cfg, budget, 8, ctx, seen, d["parent"], acc, d["k_tree"], d["v_tree"], tree,
                            d["k_cache"], d["v_cache"], score, pos, ctx2, seen2)
        ctx, seen = ctx2, seen2
        for b in range(Bq):
            n, end = int(ctx[b]), int(seen[b])
            assert n == min(budget, end)
            p = pos[:, b, :, :n].cpu().reshape(-1, n)
            for row in p.tolist():
                assert len(set(row)) == n and {0, 1} <= set(row) and set(range(end - 8, end)) <= set(row)
            for l in range(L):
                for h in range(Hkv):
                    want = every_k[l, b, pos[l, b, h, :n].cpu().long(), h]
                    assert torch.equal(d["k_cache"][l, b, :n, h].cpu(), want)


# ---- what the device refuses -------------------------------------------------------

@pytest.mark.parametrize("bad", ["parent_forward", "root_parent", "ctx_over", "ctx_negative",
                                 "accepted_over", "accepted_negative"])
def test_bad_batches_write_nothing(bad):
    inp = R.make_inputs(1, 3, 6, 4, 2, 128, 80, P=0, ctx=[80, 5, 0], seed=22)
    if bad == "parent_forward":
        inp["parent"][1, 3] = 4
    elif bad == "root_parent":
        inp["parent"][2, 0] = 0
    elif bad.startswith("ctx"):
        inp["ctx_len"][1] = 81 if bad == "ctx_over" else -1
    else:
        inp["accepted"][2] = 6 if bad == "accepted_over" else -1
    if not bad.startswith("accepted"):
        o, lse, status = run_attention(inp)
        assert status == lbx.LBX_ETREE and o.isnan().all() and lse.isnan().all()
        o, lse, status = run_attention(dict(inp, k_prefix=inp["k_cache"][:, 0], v_prefix=inp["v_cache"][:, 0]))
        assert status == lbx.LBX_ETREE and o.isnan().all() and lse.isnan().all()
    score = np.random.default_rng(0).random((1, 3, 2, 80)).astype(np.float32)
    got, tree, status = run_mass(inp, torch.zeros(1, 3, 6, 4), score)
    assert status == lbx.LBX_ETREE and np.array_equal(got, score) and np.isnan(tree).all()
    pos = np.zeros((1, 3, 2, 80), np.int32)
    (k, v, s, p, c, e), status = run_evict(inp, score, score[..., :6].copy(), pos, [80] * 3, 20, 0, 0)
    assert status == lbx.LBX_ETREE and torch.equal(k, inp["k_cache"]) and torch.equal(v, inp["v_cache"])
    assert np.array_equal(s, score) and not p.any() and (c == -7).all() and (e == -7).all()


def test_the_binding_refuses_other_shapes_types_and_layouts():
    inp = R.make_inputs(1, 2, 3, 4, 2, 64, 16, seed=23)
    cfg = cfg_of(inp)
    d = {k: v.cuda() for k, v in inp.items()}
    o, ws = torch.empty_like(d["q"]), lbx.new_cache_attn_workspace(cfg)

    def call(**kw):
        a = {**d, "o": o, **kw}
        lbx.lbx_window_attention(cfg, a["ctx_len"], a["parent"], a["q"], a["k_cache"], a["v_cache"],
                                 a["k_tree"], a["v_tree"], a["o"], ws)
    call()
    with pytest.raises(ValueError):
        call(k_cache=d["k_cache"][:, :, :8].contiguous())
    with pytest.raises(ValueError):
        call(q=d["q"].transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(TypeError):
        call(q=d["q"].half())
    with pytest.raises(TypeError):
        call(q=inp["q"])
    with pytest.raises(TypeError):
        call(ctx_len=d["ctx_len"].long())
    torch.cuda.synchronize()


def test_the_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "bounded_cache.py")
    spec = importlib.util.spec_from_file_location("bounded_cache", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    seen, ctx, o, o_win = ex.main(["--rounds", "40", "--budget", "64"])
    assert (ctx <= 64).all() and (ctx == torch.minimum(seen, torch.full_like(seen, 64))).all()
    assert (seen >= 40).all() and torch.isfinite(o).all() and torch.isfinite(o_win).all()
