"""Pins of the 64-bit definitions the cache operators' GPU tests compare with,
and the host-side refusals of their entry points (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref as R


@pytest.fixture(scope="module")
def lib():
    from tree_verify_linear_gb300 import build, lbx
    build.build()
    return lbx.load()


def test_chain_window_is_banded_causal_attention():
    """A chain over a context with a window is causal attention with a band
    and the sinks, as one dense masked softmax."""
    W, S = 7, 3
    inp = R.make_inputs(1, 1, 9, 1, 1, 64, 12, ctx=[12], tree="chain", seed=1)
    o, lse, _, _ = R.attention(inp, window=W, n_sink=S)
    k = torch.cat([inp["k_cache"], inp["k_tree"]], 2)[0, 0, :, 0].double()
    v = torch.cat([inp["v_cache"], inp["v_tree"]], 2)[0, 0, :, 0].double()
    s = inp["q"][0, 0, :, 0].double() @ k.T / 8.0
    i, j = torch.arange(12, 21)[:, None], torch.arange(21)[None]
    s[~((j <= i) & ((i - j < W) | (j < S)))] = -torch.inf
    assert np.allclose(o[0, 0, :, 0], (s.softmax(-1) @ v).numpy(), atol=1e-12)
    assert np.allclose(lse[0, 0, :, 0], s.logsumexp(-1).numpy(), atol=1e-12)


def test_window_one_sees_itself_alone():
    inp = R.make_inputs(1, 2, 5, 2, 1, 64, 6, ctx=[6, 0], seed=2)
    o, _, _, _ = R.attention(inp, window=1)
    assert np.allclose(o, inp["v_tree"].double().numpy().repeat(2, 3), atol=1e-12)


def test_prefix_equals_a_longer_cache():
    inp = R.make_inputs(1, 1, 3, 2, 2, 64, 5, P=4, ctx=[5], seed=3)
    o, lse, _, _ = R.attention(inp, prefix=True)
    flat = dict(inp, ctx_len=torch.tensor([9], dtype=torch.int32),
                k_cache=torch.cat([inp["k_prefix"][:, None], inp["k_cache"]], 2),
                v_cache=torch.cat([inp["v_prefix"][:, None], inp["v_cache"]], 2))
    o2, lse2, _, _ = R.attention(flat)
    assert np.allclose(o, o2, atol=1e-12) and np.allclose(lse, lse2, atol=1e-12)


def test_masses_of_a_path_sum_to_its_queries():
    """Every query's weights sum to one."""
    inp = R.make_inputs(2, 2, 8, 6, 2, 64, 20, seed=4)
    _, lse, _, _ = R.attention(inp)
    score, tree, _, _ = R.mass(inp, lse, np.zeros((2, 2, 2, 20), np.float32))
    for b in range(2):
        path = R.root_path(inp["parent"][b].tolist(), int(inp["accepted"][b]))
        assert np.allclose(score[:, b].sum(-1) + tree[:, b].sum(-1), 3 * len(path), atol=1e-10)
        off = [n for n in range(8) if n not in path]
        assert not tree[:, b][..., off].any()


def test_evict_worked_by_hand():
    """Five entries of scores 5 1 4 1 3, one new of score 2, four stay: entries
    0, 2, 4 and the new one; 4 and the new one take places 1 and 3."""
    inp = R.make_inputs(1, 1, 1, 1, 1, 64, 6, ctx=[5], seed=5)
    score = np.array([5, 1, 4, 1, 3, 9], np.float32).reshape(1, 1, 1, 6)
    pos = np.arange(6, dtype=np.int32).reshape(1, 1, 1, 6)
    k, v, s, p, ctx, seen = R.evict(inp, score, np.full((1, 1, 1, 1), 2, np.float32), pos, [5], 4, 0, 0)
    assert s[0, 0, 0, :4].tolist() == [5, 3, 4, 2] and p[0, 0, 0, :4].tolist() == [0, 4, 2, 5]
    assert ctx.tolist() == [4] and seen.tolist() == [6]
    assert torch.equal(k[0, 0, 1], inp["k_cache"][0, 0, 4]) and torch.equal(v[0, 0, 3], inp["v_tree"][0, 0, 0])


GOOD = dict(L=1, Bq=1, N=4, Hq=4, Hkv=2, dh=64, T=8)


@pytest.mark.parametrize("change", [
    dict(L=0), dict(Bq=0), dict(N=0), dict(N=65), dict(Hkv=3), dict(Hkv=0), dict(dh=96), dict(dh=32),
    dict(T=-1), dict(P=-1), dict(window=-1), dict(n_sink=-1), dict(dtype=2), dict(scale=0.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(L=1 << 15, Bq=1 << 15)])
def test_bad_configs_are_refused(lib, change):
    from tree_verify_linear_gb300 import lbx
    assert lbx.lbx_cache_attn_workspace_size(lbx.make_attn_cfg(**GOOD)) > 0
    cfg = lbx.make_attn_cfg(**{**GOOD, **change})
    assert lbx.lbx_cache_attn_workspace_size(cfg) == 0
    with pytest.raises(lbx.LbxError):
        lbx.new_cache_attn_workspace(cfg)
    r, p = ctypes.byref(cfg), ctypes.c_void_p(1 << 20)  # aligned, never read: refused first
    assert lib.lbx_window_attention(r, *[p] * 9, p, 1 << 40, None, None) == lbx.LBX_EINVAL
    cfg.P = cfg.P or 4
    assert lib.lbx_prefix_attention(r, *[p] * 11, p, 1 << 40, None, None) == lbx.LBX_EINVAL
    cfg.P = 0 if change != dict(P=-1) else -1
    assert lib.lbx_attention_mass(r, *[p] * 9, None, None) == lbx.LBX_EINVAL
    assert lib.lbx_cache_evict(r, 4, 0, *[p] * 13, None, None) == lbx.LBX_EINVAL


def test_bad_pointers_and_arguments_are_refused(lib):
    from tree_verify_linear_gb300 import lbx
    good, ws = ctypes.c_void_p(1 << 20), 1 << 40
    cfg = lbx.make_attn_cfg(**GOOD)
    r = ctypes.byref(cfg)

    def each_bad(n, call):
        for i in range(n):
            for bad in (None, ctypes.c_void_p((1 << 20) + 2)):
                args = [good] * n
                args[i] = bad
                if call(args) != lbx.LBX_EINVAL:
                    return i
        return None
    # lse (the last) may be NULL: tested apart
    assert each_bad(8, lambda a: lib.lbx_window_attention(r, *a, None, good, ws, None, None)) is None
    odd = ctypes.c_void_p((1 << 20) + 2)
    assert lib.lbx_window_attention(r, *[good] * 8, odd, good, ws, None, None) == lbx.LBX_EINVAL
    assert lib.lbx_window_attention(r, *[good] * 9, None, ws, None, None) == lbx.LBX_EINVAL
    assert lib.lbx_window_attention(r, *[good] * 9, good, 0, None, None) == lbx.LBX_EINVAL
    assert lib.lbx_window_attention(r, *[good] * 9, good, ws, odd, None) == lbx.LBX_EINVAL
    assert each_bad(9, lambda a: lib.lbx_attention_mass(r, *a, None, None)) is None
    assert lib.lbx_attention_mass(r, *[good] * 9, odd, None) == lbx.LBX_EINVAL
    assert each_bad(13, lambda a: lib.lbx_cache_evict(r, 4, 0, *a, None, None)) is None
    for budget, recent in ((0, 0), (9, 0), (4, -1)):
        assert lib.lbx_cache_evict(r, budget, recent, *[good] * 13, None, None) == lbx.LBX_EINVAL
    # a prefix belongs to lbx_prefix_attention, a window to lbx_window_attention
    assert lib.lbx_prefix_attention(r, *[good] * 11, good, ws, None, None) == lbx.LBX_EINVAL
    cfg.P = 4
    assert each_bad(10, lambda a: lib.lbx_prefix_attention(r, *a, None, good, ws, None, None)) is None
    assert lib.lbx_window_attention(r, *[good] * 9, good, ws, None, None) == lbx.LBX_EINVAL
    cfg.window = 3
    assert lib.lbx_prefix_attention(r, *[good] * 11, good, ws, None, None) == lbx.LBX_EINVAL
    long_cfg = lbx.make_attn_cfg(**{**GOOD, "T": lbx.LBX_EVICT_MAX_T + 1})
    assert lib.lbx_cache_evict(ctypes.byref(long_cfg), 4, 0, *[good] * 13, None, None) == lbx.LBX_EINVAL
