"""GPU tests of the bounded cache's operators at their edges: full windows,
shared workspaces, calls side by side, NaN, the longest windows."""
import numpy as np
import pytest
import torch

import cache_ref as R
from test_gpu_cache import (built, cfg_of, check_attention, run_attention, run_evict,  # noqa: F401
                            run_mass)  # (built: a fixture)
from tree_verify_linear_gb300 import lbx

pytestmark = pytest.mark.gpu


# ---- a window as long as a full cache ---------------------------------------

@pytest.mark.parametrize("T,n_sink", [(2, 1), (64, 1), (64, 64), (65, 4), (100, 4), (128, 70), (512, 4), (1024, 1)])
@pytest.mark.parametrize("dh,dtype,N,Hq", [(64, "f16", 1, 1), (128, "bf16", 1, 4), (256, "bf16", 3, 5)])
def test_window_as_long_as_a_full_cache(T, n_sink, dh, dtype, N, Hq):
    """Its first position is past the window and a first position that stays
    visible; twice on one workspace."""
    inp = R.make_inputs(1, 2, N, Hq, 1, dh, T, dtype=dtype, ctx=[T, T - 1], seed=T + n_sink)
    o, lse = check_attention(inp, window=T, n_sink=n_sink)
    o2, lse2, status = run_attention(inp, calls=2, window=T, n_sink=n_sink)
    assert status == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


# ---- the longest windows ------------------------------------------------------

@pytest.mark.parametrize("dh,T", [(64, 30), (128, 2000), (256, 70)])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 40])
def test_the_longest_windows_are_no_window(dh, T, window):
    inp = R.make_inputs(1, 2, 40, 4, 2, dh, T, ctx=[T, T // 2], tree="chain", seed=dh)
    inp["accepted"][:] = 39
    o, lse, _ = run_attention(inp)
    o2, lse2, status = run_attention(inp, window=window)
    assert status == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    score = np.zeros((1, 2, 2, T), np.float32)
    s, tree, _ = run_mass(inp, lse, score)
    s2, tree2, status = run_mass(inp, lse, score, window=window)
    assert status == 0 and np.array_equal(s, s2) and np.array_equal(tree, tree2)


# ---- the first segment of a block of threads -----------------------------------

@pytest.mark.parametrize("dh,N,Hq,T,dtype", [(256, 22, 6, 0, "bf16"), (128, 64, 4, 1, "f16"), (64, 40, 3, 0, "bf16")])
def test_every_request_reads_its_own_tree(dh, N, Hq, T, dtype):
    """As many requests as multiprocessors, each with a tree of its own and next to
    no cache: every block of threads begins with another tree's masks."""
    inp = R.make_inputs(1, 152, N, Hq, 1, dh, T, dtype=dtype, seed=dh + N)
    o, lse, status = run_attention(inp)
    assert status == 0
    ref_o, ref_lse, o_tol, lse_tol = R.attention_dense(inp)
    assert (np.abs(o.double().numpy() - ref_o) <= o_tol).all()
    assert (np.abs(lse.double().numpy() - ref_lse) <= lse_tol).all()
    o2, lse2, status = run_attention(inp, calls=200)
    assert status == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


# ---- one workspace for many configurations ---------------------------------------

def test_calls_of_every_kind_take_turns_on_one_workspace():
    """Batch sizes, head dimensions, with and without a prefix, streams in many
    pieces and the small kernel: each call gives what it gives on a workspace of its own."""
    kinds = [(dict(L=4, Bq=b, N=22, Hq=12, Hkv=2, dh=256, T=700, P=p, dtype=t), {})
             for b, p, t in ((4, 900, "bf16"), (5, 900, "bf16"), (3, 0, "f16"), (6, 0, "bf16"))]
    kinds += [(dict(L=1, Bq=b, N=12, Hq=4, Hkv=1, dh=dh, T=9000, P=p), {})
              for b, dh, p in ((1, 64, 0), (2, 128, 0), (7, 64, 5000), (1, 256, 3000))]
    kinds += [(dict(L=1, Bq=2, N=1, Hq=8, Hkv=4, dh=dh, T=500, P=p), {}) for dh, p in ((64, 0), (256, 100))]
    kinds += [(dict(L=2, Bq=3, N=5, Hq=8, Hkv=2, dh=128, T=3000), dict(window=900, n_sink=4))]
    calls = []
    for i, (sizes, kw) in enumerate(kinds):
        inp = R.make_inputs(**sizes, seed=600 + i)
        o, lse, status = run_attention(inp, **kw)
        assert status == 0
        calls.append((cfg_of(inp, **kw), {k: v.cuda() for k, v in inp.items()}, o.cuda(), lse.cuda()))
    ws = torch.zeros(max(lbx.lbx_cache_attn_workspace_size(c[0]) for c in calls), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(3 * len(calls)):
        cfg, d, o, lse = calls[step * 5 % len(calls)]
        got, got_lse = torch.full_like(o, float("nan")), torch.full_like(lse, float("nan"))
        pre = (d["k_prefix"], d["v_prefix"]) if cfg.P else ()
        (lbx.lbx_prefix_attention if cfg.P else lbx.lbx_window_attention)(
            cfg, d["ctx_len"], d["parent"], d["q"], *pre, d["k_cache"], d["v_cache"], d["k_tree"],
            d["v_tree"], got, ws, lse=got_lse, d_status=status)
        assert torch.equal(got, o) and torch.equal(got_lse, lse), step
    assert int(status.item()) == 0 and not ws[:4096].any()


# ---- calls side by side ------------------------------------------------------------

@pytest.mark.parametrize("P", [0, 9000])
def test_calls_on_streams_of_two_priorities(P):
    """Streams cut into pieces for every multiprocessor, two calls at a time: the
    one of higher priority takes the multiprocessors that the other's blocks wait for.
    Neither may depend on a block that is not running."""
    inps = [R.make_inputs(L=1, Bq=2, N=22, Hq=6, Hkv=1, dh=256, T=500 if P else 9000, P=P,
                          ctx=[500, 0] if P else [9000, 7000], seed=700),
            R.make_inputs(L=1, Bq=1, N=3, Hq=8, Hkv=1, dh=128, T=20000, dtype="f16", ctx=[19999], seed=701)]
    calls = []
    for inp, priority in zip(inps, (0, -1)):
        o, lse, status = run_attention(inp)
        assert status == 0
        cfg = cfg_of(inp)
        calls.append((cfg, {k: v.cuda() for k, v in inp.items()}, o.cuda(), lse.cuda(),
                      lbx.new_cache_attn_workspace(cfg), torch.cuda.Stream(priority=priority)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [[(torch.full_like(c[2], float("nan")), torch.empty_like(c[3])) for c in calls] for _ in range(20)]
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record()
    for turn in outs:
        for (cfg, d, _, _, ws, stream), (o, lse) in zip(calls, turn):
            pre = (d["k_prefix"], d["v_prefix"]) if cfg.P else ()
            (lbx.lbx_prefix_attention if cfg.P else lbx.lbx_window_attention)(
                cfg, d["ctx_len"], d["parent"], d["q"], *pre, d["k_cache"], d["v_cache"], d["k_tree"],
                d["v_tree"], o, ws, lse=lse, d_status=status, stream=stream)
    torch.cuda.synchronize()
    end.record()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for turn in outs:
        for (_, _, o, lse, _, _), (got, got_lse) in zip(calls, turn):
            assert torch.equal(got, o) and torch.equal(got_lse, lse)
    assert begin.elapsed_time(end) < 1000  # a wait for a block that cannot run would take seconds


# ---- NaN that a query does see -------------------------------------------------------

NAN = {  # streams whole, in two pieces, in many, joined with a prefix's; the small kernel
    "whole_pair": dict(L=16, Bq=6, N=22, Hq=12, Hkv=2, dh=256, T=200, ctx=[200] * 6),
    "whole": dict(L=16, Bq=12, N=5, Hq=4, Hkv=1, dh=64, T=300, dtype="f16", ctx=[300] * 12),
    "two_pieces": dict(L=1, Bq=1, N=22, Hq=48, Hkv=8, dh=256, T=4500, ctx=[4500]),
    "many_pieces_pair": dict(L=1, Bq=2, N=22, Hq=6, Hkv=1, dh=256, T=9000, ctx=[9000, 8000]),
    "many_pieces": dict(L=1, Bq=2, N=12, Hq=4, Hkv=1, dh=64, T=20000, ctx=[19999, 7000]),
    "prefix_pair": dict(L=2, Bq=5, N=22, Hq=12, Hkv=2, dh=128, T=300, P=3001, dtype="f16", ctx=[300] * 5),
    "prefix": dict(L=1, Bq=40, N=2, Hq=16, Hkv=4, dh=64, T=300, P=2049, ctx=[300] * 40),
    "few_one_unit": dict(L=1, Bq=2, N=3, Hq=4, Hkv=2, dh=128, T=0),
    "few_units": dict(L=1, Bq=2, N=1, Hq=8, Hkv=2, dh=256, T=700, ctx=[700, 650]),
    "few_prefix": dict(L=1, Bq=2, N=2, Hq=4, Hkv=2, dh=64, T=90, P=150, dtype="f16", ctx=[90, 90]),
}


@pytest.mark.parametrize("name", sorted(NAN))
def test_a_nan_score_makes_its_query_nan(name):
    inp = R.make_inputs(**NAN[name], seed=800 + len(name))
    o, lse, _ = run_attention(inp)
    nan = float("nan")
    L, Bq, N, Hq = lse.shape
    G, T = Hq // inp["k_tree"].shape[3], inp["k_cache"].shape[2]

    def check(change, rows, lse_too=True):
        bad = {k: v.clone() for k, v in inp.items()}
        change(bad)
        o2, lse2, status = run_attention(bad)
        assert status == 0
        hit = torch.zeros(lse.shape, dtype=torch.bool)
        hit[rows] = True
        assert o2[hit].isnan().all() and torch.equal(o2[~hit], o[~hit])
        want = torch.where(hit, torch.full_like(lse, nan), lse) if lse_too else lse
        assert torch.equal(torch.nan_to_num(lse2, nan=1e30), torch.nan_to_num(want, nan=1e30))

    def one(bad, key, *at):
        bad[key][at] = nan
    # a query; the root's key; a cached key, the first and the last; one of the prefix; a value
    check(lambda d: one(d, "q", L - 1, Bq - 1, N - 1, Hq - 1, 3), (L - 1, Bq - 1, N - 1, Hq - 1))
    check(lambda d: one(d, "k_tree", 0, 0, 0, 0, 0), (0, 0, slice(None), slice(G)))
    if T:
        for j in (0, int(inp["ctx_len"][0]) - 1):
            check(lambda d: one(d, "k_cache", 0, 0, j, 0, 1), (0, 0, slice(None), slice(G)))
        check(lambda d: one(d, "v_cache", 0, 0, T // 3, 0), (0, 0, slice(None), slice(G)), lse_too=False)
    if "k_prefix" in inp:
        check(lambda d: one(d, "k_prefix", 0, 77, 0, 0), (0, slice(None), slice(None), slice(G)))


def test_nan_beside_a_prefix_without_a_finite_score():
    """Neither side's -inf hides the other's NaN."""
    inp = R.make_inputs(1, 40, 2, 16, 4, 64, 30, P=2049, ctx=[30] * 40, seed=31)
    inp["q"] = inp["q"].abs() + 1
    for finite, hidden in ((("k_prefix",), ("k_cache", "k_tree")), (("k_cache", "k_tree"), ("k_prefix",))):
        bad = {k: v.clone() for k, v in inp.items()}
        for k in finite:
            bad[k][:] = -float("inf")
        for k in hidden:
            bad[k][:] = float("nan")
        o, lse, status = run_attention(bad)
        assert status == 0 and o.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_a_nan_lse_reaches_the_weights_of_the_keys_it_sees(dh):
    inp = R.make_inputs(1, 2, 8, 4, 2, dh, 150, ctx=[150, 90], tree="chain", seed=32)
    inp["accepted"][:] = 7
    _, ref_lse, _, _ = R.attention(inp, window=40, n_sink=2)
    lse = torch.from_numpy(ref_lse.astype(np.float32))
    score = np.zeros((1, 2, 2, 150), np.float32)
    clean, clean_tree, _ = run_mass(inp, lse, score, window=40, n_sink=2)
    lse[0, 0, 5, 0] = float("nan")
    got, tree, status = run_mass(inp, lse, score, window=40, n_sink=2)
    assert status == 0
    js, ms = R.visible(inp["parent"][0].tolist(), 5, 150, 40, 2)
    hit, hit_tree = np.zeros(got.shape, bool), np.zeros(tree.shape, bool)
    hit[0, 0, 0, js], hit_tree[0, 0, 0, ms] = True, True
    assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], clean[~hit])
    assert np.isnan(tree[hit_tree]).all() and np.array_equal(tree[~hit_tree], clean_tree[~hit_tree])


# ---- windows and eviction ----------------------------------------------------------

def test_the_example_windows_see_the_last_positions():
    """Its windowed queries see the positions up to their own, of a cache that
    holds them all in order, while the other cache drops entries."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "bounded_cache.py")
    spec = importlib.util.spec_from_file_location("bounded_cache", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    s = ex.serve(60, 64)
    n = s["seen"].tolist()
    assert s["len_all"].tolist() == n and (s["ctx"] == 64).all() and min(n) > ex.WINDOW
    for b in range(ex.BQ):
        assert (s["pos_all"][:, b, :, :n[b]].cpu() == torch.arange(n[b])).all()
    inp = {k: s[k].cpu() for k in ("parent", "q", "k_tree", "v_tree", "ctx_len")}
    inp.update(k_cache=s["k_all"].cpu(), v_cache=s["v_all"].cpu())
    ref, _, tol, _ = R.attention_dense(inp, window=ex.WINDOW, n_sink=ex.SINKS)
    assert (np.abs(s["o_win"].cpu().double().numpy() - ref) <= tol).all()


# ---- host threads --------------------------------------------------------------------

def test_host_threads_call_with_different_sizes():
    """Two threads, small and large calls of the operators whose shared memory goes
    by their sizes; the library lets them run at the same time."""
    import threading
    ok, failed = [], []

    def work(T, N):
        try:
            inp = R.make_inputs(1, 1, N, 8, 1, 64, T, ctx=[T], seed=T)
            d = {k: v.cuda() for k, v in inp.items()}
            cfg, stream = cfg_of(inp), torch.cuda.Stream()
            f32, i32 = {"device": "cuda"}, {"dtype": torch.int32, "device": "cuda"}
            lse, score, tree = torch.zeros(1, 1, N, 8, **f32), torch.zeros(1, 1, 1, T, **f32), torch.zeros(1, 1, 1, N, **f32)
            pos, outs = torch.zeros(1, 1, 1, T, **i32), [torch.zeros(1, **i32) for _ in range(2)]
            torch.cuda.synchronize()
            for _ in range(1500):
                lbx.lbx_attention_mass(cfg, d["ctx_len"], d["parent"], d["accepted"], d["q"], lse,
                                       d["k_cache"], d["k_tree"], score, tree, stream=stream)
                lbx.lbx_cache_evict(cfg, T, 0, d["ctx_len"], d["ctx_len"], d["parent"], d["accepted"],
                                    d["k_tree"], d["v_tree"], tree, d["k_cache"], d["v_cache"], score,
                                    pos, *outs, stream=stream)
            stream.synchronize()
            ok.append(T)
        except Exception as e:  # noqa: BLE001 (told to the test's own thread)
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=a) for a in ((70, 1), (15000, 30), (1000, 8))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(ok) == 3, failed


def test_the_longest_cache_evict_takes():
    T = lbx.LBX_EVICT_MAX_T
    inp = R.make_inputs(1, 1, 64, 1, 1, 64, T, ctx=[T], tree="chain", seed=33)
    inp["accepted"][:] = 63
    score = np.arange(T, dtype=np.float32).reshape(1, 1, 1, T)
    pos = np.arange(T, dtype=np.int32).reshape(1, 1, 1, T)
    tree = np.full((1, 1, 1, 64), 2.0 * T, np.float32)
    (k, v, s, p, ctx, seen), status = run_evict(inp, score, tree, pos, [T], T, 0, 0)
    # the 64 lowest leave, the path takes their places in order
    assert status == 0 and ctx.tolist() == [T] and seen.tolist() == [T + 64]
    assert p[0, 0, 0, :64].tolist() == list(range(T, T + 64)) and np.array_equal(p[..., 64:], pos[..., 64:])
    assert torch.equal(k[0, 0, :64], inp["k_tree"][0, 0]) and torch.equal(v[:, :, 64:], inp["v_cache"][:, :, 64:])


def test_eviction_takes_outputs_beside_its_inputs():
    """ctx_len, seen, accepted and the outputs as rows of one array."""
    Bq = 16
    inp = R.make_inputs(1, Bq, 3, 2, 2, 64, 40, seed=34)
    d = {k: v.cuda() for k, v in inp.items()}
    rows = torch.zeros(5, Bq, dtype=torch.int32, device="cuda")
    rows[0], rows[1], rows[2] = d["ctx_len"], 50, d["accepted"]
    score = torch.rand(1, Bq, 2, 40, device="cuda")
    pos = torch.zeros(1, Bq, 2, 40, dtype=torch.int32, device="cuda")
    args = (d["parent"], rows[2], d["k_tree"], d["v_tree"], torch.rand(1, Bq, 2, 3, device="cuda"),
            d["k_cache"], d["v_cache"], score, pos)
    lbx.lbx_cache_evict(cfg_of(inp), 30, 0, rows[0], rows[1], *args, rows[3], rows[4])
    for b in range(Bq):
        path = len(R.root_path(inp["parent"][b].tolist(), int(inp["accepted"][b])))
        assert rows[3, b] == min(30, int(inp["ctx_len"][b]) + path) and rows[4, b] == 50 + path
    with pytest.raises(lbx.LbxError):
        lbx.lbx_cache_evict(cfg_of(inp), 30, 0, rows[0], rows[1], *args, rows[0], rows[4])


# ---- many small weights beside a large one ---------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dh,N,Hq,Bq,T", [(64, 1, 1, 160, 8192), (128, 44, 3, 80, 4096), (256, 1, 1, 160, 4096)])
def test_many_small_weights_beside_a_large_one(dtype, dh, N, Hq, Bq, T):
    """The first key scores 17.75 above all others, whose weights (2^-25.6) are below
    the smallest f16: together they are all there is of o, whose error is the
    roundings of o and of the weights (u each) and, in f16, 2^-32 for each key."""
    el = R.DTYPE[dtype]
    q = torch.zeros(1, Bq, N, Hq, dh, dtype=el, device="cuda")
    q[..., 0] = 8
    kc, vc = (torch.zeros(1, Bq, T, 1, dh, dtype=el, device="cuda") for _ in range(2))
    kc[:, :, 0, :, 0], vc[:, :, 1:] = 17.75, 1
    kt, vt = (torch.zeros(1, Bq, N, 1, dh, dtype=el, device="cuda") for _ in range(2))
    kt[..., 0] = -100
    parent = torch.zeros(Bq, N, dtype=torch.int32, device="cuda")
    parent[:, 0] = -1
    ctx, status = torch.full((Bq,), T, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg = lbx.make_attn_cfg(1, Bq, N, Hq, 1, dh, T, dtype=lbx.LBX_F16 if dtype == "f16" else lbx.LBX_BF16, scale=0.125)
    o, lse = torch.empty_like(q), torch.empty(1, Bq, N, Hq, device="cuda")
    lbx.lbx_window_attention(cfg, ctx, parent, q, kc, vc, kt, vt, o, lbx.new_cache_attn_workspace(cfg), lse=lse,
                             d_status=status)
    small = (T - 1) * np.exp(-17.75)
    want, u = small / (1 + small), 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    tol = 2 * u * want + (T * 2.0 ** -32 if dtype == "f16" else 0)
    assert int(status.item()) == 0 and float((o.double() - want).abs().max()) <= tol
    assert float((lse.double() - 17.75 - np.log1p(small)).abs().max()) <= 2.0 ** -20 * 20


# ---- full-context tree attention ---------------------------------------------------------

def test_tree_attention_gives_the_same_bits_every_time():
    """Its halves of a row exchange every block's maxima: two buffers, so that one
    may run ahead of the other; 200 calls of 64 blocks per block of threads agree."""
    L, Bq, N, Hq, Hkv, dh, T = 2, 3, 22, 12, 2, 256, 20000
    inp = R.make_inputs(L, Bq, N, Hq, Hkv, dh, T, ctx=[20000, 17001, 19], seed=35)
    d = {k: v.cuda() for k, v in inp.items()}
    ws = lbx.new_attn_workspace(L, Bq, N, Hq, Hkv, dh, T)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.empty(L, Bq, N, Hq, dh, device="cuda") for _ in range(2)]
    for i in range(200):
        lbx.lbx_tree_attention(dh ** -0.5, d["ctx_len"], d["parent"], d["q"], d["k_cache"], d["v_cache"],
                               d["k_tree"], d["v_tree"], outs[min(i, 1)], ws, status)
        if i:
            assert torch.equal(outs[0], outs[1]), i
    ref, _, tol, _ = R.attention_dense(inp)
    assert int(status.item()) == 0 and (np.abs(outs[0].cpu().double().numpy() - ref) <= tol).all()


# ---- precision of the weights ---------------------------------------------------------

@pytest.mark.parametrize("dh,N,Hq,Bq", [(64, 1, 1, 100), (64, 1, 1, 400), (128, 1, 2, 400), (128, 43, 3, 200),
                                        (256, 1, 1, 100), (256, 1, 1, 400), (256, 22, 6, 200)])
def test_bf16_weights_are_not_rounded_to_bf16(dh, N, Hq, Bq):
    """Two keys whose values nearly cancel: o is what the rounding of the second value
    leaves, 2^-8 of a weight at most.  Weights in bf16 would be off by as much; as hi + lo
    they are good to 2^-17, and o's own rounding is 2^-8 of o.  (e: of a score, as in
    cache_ref; every row of a request asks the same.)"""
    g = torch.Generator().manual_seed(dh + N)
    q0 = torch.randn(Bq, dh, generator=g).bfloat16()
    k = torch.randn(Bq, 2, dh, generator=g).bfloat16()
    q0[:, 0], k[:, :, 0] = 8, 0
    s = torch.einsum("bd,bjd->bj", q0.double(), k.double()) * dh ** -0.5
    w = s.softmax(-1)
    v1 = (-(w[:, 0] / w[:, 1])).bfloat16()
    want = w[:, 0] + w[:, 1] * v1.double()
    e = (dh + 2) * 2.0 ** -24 * dh ** -0.5 * torch.einsum("bd,bjd->bj", q0.double().abs(), k.double().abs()).amax(-1)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -17 + 2 * e + 2.0 ** -20) * 2 * w[:, 0]
    inp = {"q": q0[None, :, None, None].expand(1, Bq, N, Hq, dh).contiguous(), "k_cache": k[None, :, :, None],
           "v_cache": torch.stack([torch.ones_like(v1), v1], 1)[None, :, :, None, None].expand(1, Bq, 2, 1, dh).contiguous(),
           "k_tree": torch.zeros(1, Bq, N, 1, dh).bfloat16(), "v_tree": torch.zeros(1, Bq, N, 1, dh).bfloat16(),
           "ctx_len": torch.full((Bq,), 2, dtype=torch.int32), "parent": torch.zeros(Bq, N, dtype=torch.int32)}
    inp["k_tree"][..., 0] = -1000
    inp["parent"][:, 0] = -1
    o, _, status = run_attention(inp)
    over = (o[0].double() - want[:, None, None, None]).abs() / tol[:, None, None, None]
    assert status == 0 and float(over.max()) <= 1


# ---- single tokens in f16 ---------------------------------------------------------------

@pytest.mark.parametrize("dh", [64, 128, 256])
@pytest.mark.parametrize("Bq,T,window", [(2, 1, 0), (2, 65, 0), (3, 300, 100), (16, 2100, 0), (16, 2500, 700)])
def test_single_tokens_in_f16(dh, Bq, T, window):
    """Attention and weights of plain decode steps, the small kernel's and the large one's."""
    inp = R.make_inputs(2, Bq, 1, 8, 4, dh, T, dtype="f16", seed=dh + T)
    o, lse, status = run_attention(inp, window=window, n_sink=3)
    assert status == 0
    ref_o, ref_lse, o_tol, lse_tol = R.attention_dense(inp, window=window, n_sink=3)
    assert (np.abs(o.double().numpy() - ref_o) <= o_tol).all()
    assert (np.abs(lse.double().numpy() - ref_lse) <= lse_tol).all()
    score = np.random.default_rng(3).random((2, Bq, 4, T)).astype(np.float32)
    got, tree, status = run_mass(inp, lse, score, window=window, n_sink=3)
    ref, ref_tree, tol, tree_tol = R.mass(inp, lse.numpy(), score, window=window, n_sink=3)
    assert status == 0 and (np.abs(got - ref) <= tol).all() and (np.abs(tree - ref_tree) <= tree_tol).all()


# ---- the current stream --------------------------------------------------------------------

def test_calls_go_to_the_current_stream(monkeypatch):
    """With torch's quick way to its handle, and without it."""
    t, side = torch.zeros(1, device="cuda"), torch.cuda.Stream()
    for quick in (True, False):
        if not quick:
            monkeypatch.setattr(lbx, "_raw_stream", lbx._public_raw_stream)
        assert lbx._stream_of(t, None) == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(side):
            assert lbx._stream_of(t, None) == side.cuda_stream
        assert lbx._stream_of(t, side) == side.cuda_stream
    inp = R.make_inputs(1, 2, 3, 4, 2, 64, 50, seed=36)
    o, lse, _ = run_attention(inp)
    with torch.cuda.stream(side):
        o2, lse2, status = run_attention(inp)
    assert status == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


# ---- graphs --------------------------------------------------------------------------------

@pytest.mark.parametrize("sizes", [dict(L=1, Bq=2, N=1, Hq=8, Hkv=2, dh=128, T=200),
                                   dict(L=2, Bq=3, N=22, Hq=12, Hkv=2, dh=256, T=700),
                                   dict(L=1, Bq=6, N=22, Hq=6, Hkv=1, dh=256, T=300, P=9000),
                                   dict(L=1, Bq=40, N=2, Hq=16, Hkv=4, dh=64, T=300, P=2049, dtype="f16")])
def test_a_round_of_calls_replays_from_a_graph(sizes):
    """Attention, weights and eviction captured together, replayed on new lengths."""
    inp = R.make_inputs(**sizes, seed=37)
    cfg = cfg_of(inp)
    d = {k: v.cuda() for k, v in inp.items()}
    L, Bq, N, Hq, T = *inp["q"].shape[:4], cfg.T
    ws, status = lbx.new_cache_attn_workspace(cfg), torch.zeros(1, dtype=torch.int32, device="cuda")
    seen = torch.full((Bq,), 3 * T, dtype=torch.int32, device="cuda")
    pre = (d["k_prefix"], d["v_prefix"]) if cfg.P else ()
    start = {"k_cache": d["k_cache"].clone(), "v_cache": d["v_cache"].clone(),
             "score": torch.rand(L, Bq, cfg.Hkv, T, device="cuda"),
             "pos": torch.randint(3 * T, (L, Bq, cfg.Hkv, T), dtype=torch.int32, device="cuda")}
    s = {k: v.clone() for k, v in start.items()}
    s.update(o=torch.empty_like(d["q"]), lse=torch.empty(L, Bq, N, Hq, device="cuda"),
             tree=torch.empty(L, Bq, cfg.Hkv, N, device="cuda"), ctx_out=torch.empty_like(seen), seen_out=torch.empty_like(seen))

    def calls():
        (lbx.lbx_prefix_attention if cfg.P else lbx.lbx_window_attention)(
            cfg, d["ctx_len"], d["parent"], d["q"], *pre, s["k_cache"], s["v_cache"], d["k_tree"], d["v_tree"],
            s["o"], ws, lse=s["lse"], d_status=status)
        lbx.lbx_attention_mass(cfg, d["ctx_len"], d["parent"], d["accepted"], d["q"], s["lse"], s["k_cache"],
                               d["k_tree"], s["score"], s["tree"], d_status=status)
        lbx.lbx_cache_evict(cfg, T // 2, 5, d["ctx_len"], seen, d["parent"], d["accepted"], d["k_tree"], d["v_tree"],
                            s["tree"], s["k_cache"], s["v_cache"], s["score"], s["pos"], s["ctx_out"], s["seen_out"],
                            d_status=status)

    def reset():
        for k, v in start.items():
            s[k].copy_(v)
    calls()
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for ctx in ([T] * Bq, [b * T // Bq for b in range(Bq)], [0] * Bq):
        d["ctx_len"].copy_(torch.tensor(ctx, dtype=torch.int32))
        reset()
        calls()
        want = {k: v.clone() for k, v in s.items()}
        reset()
        graph.replay()
        for k, v in s.items():
            assert torch.equal(v, want[k]), (k, ctx)
    assert int(status.item()) == 0
