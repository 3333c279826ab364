"""Thin Python binding of the liblbx C ABI (include/lbx.h).

Argument marshalling only: every step of the verify path runs in the CUDA
kernels of liblbx.so.  The functions keep the C names and argument order and
take torch CUDA tensors (PyTorch supplies device memory and streams).  bf16
arguments may be ``torch.bfloat16`` or 16-bit integer tensors holding bf16 bit
patterns.  There is no CPU fallback: if the library cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblbx.so")

LBX_OK, LBX_EINVAL, LBX_ECUDA, LBX_ETREE, LBX_ETIMEOUT, LBX_EPAGES = 0, -1, -2, -3, -4, -5
LBX_MAX_TREE_NODES = 64
LBX_CHAIN_CHUNK = 64
LBX_MAX_CONV_WIDTH = 4
LBX_MODE_AUTO, LBX_MODE_TREE, LBX_MODE_CHUNKED, LBX_MODE_TREE_CUDA_CORES = 0, 1, 2, 3

# Every function the header declares, in header order.
EXPORTS = ("lbx_strerror", "lbx_workspace_size", "lbx_tree_conv", "lbx_tree_deltanet",
           "lbx_tree_persist", "lbx_verify_step", "lbx_verify_step_noalloc",
           "lbx_accept_workspace_size", "lbx_accept_walk", "lbx_ddtree_build",
           "lbx_attn_workspace_size", "lbx_tree_attention", "lbx_cache_attn_workspace_size",
           "lbx_window_attention", "lbx_prefix_attention", "lbx_attention_mass",
           "lbx_cache_evict", "lbx_page_tables", "lbx_qk_norm_rope", "lbx_paged_workspace_size",
           "lbx_paged_attention", "lbx_page_commit")
LBX_ACCEPT_MAX_NODES = 4096
LBX_DDTREE_MAX_K, LBX_DDTREE_MAX_DEPTH = 8, 64
LBX_NOALLOC_MAX_GROUPS = 65536
LBX_ATTN_HEAD_DIM, LBX_ATTN_MAX_NODES = 256, 64
LBX_BF16, LBX_F16 = 0, 1
LBX_EVICT_MAX_T = 1 << 20
LBX_PAGE_MAX_REQUESTS, LBX_PAGED_MAX_GROUP = 2048, 128
LBX_ROPE_HALVES, LBX_ROPE_ADJACENT, LBX_ROPE_MAX_AXES = 0, 1, 4
LBX_WEIGHTS_ROUNDED, LBX_WEIGHTS_SPLIT = 0, 1


class LbxError(RuntimeError):
    def __init__(self, fn: str, rc: int):
        super().__init__(f"{fn} failed: {rc} ({strerror(rc)})")
        self.rc = rc


class lbx_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("Bq", ctypes.c_int), ("N", ctypes.c_int),
                ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("d", ctypes.c_int),
                ("K", ctypes.c_int), ("n_slots", ctypes.c_int), ("l2_eps", ctypes.c_float),
                ("q_scale", ctypes.c_float), ("mode", ctypes.c_int)]


class lbx_attn_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("Bq", ctypes.c_int), ("N", ctypes.c_int),
                ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("dh", ctypes.c_int),
                ("T", ctypes.c_int), ("P", ctypes.c_int), ("window", ctypes.c_int),
                ("n_sink", ctypes.c_int), ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


class lbx_page_cfg(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int), ("Bq", ctypes.c_int), ("M", ctypes.c_int),
                ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("dh", ctypes.c_int),
                ("page", ctypes.c_int), ("n_pages", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("weights", ctypes.c_int)]


class lbx_rope_cfg(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("axes", ctypes.c_int),
                ("section", ctypes.c_int * LBX_ROPE_MAX_AXES), ("pairing", ctypes.c_int),
                ("eps", ctypes.c_float)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblbx.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"liblbx.so not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        lib.lbx_strerror.restype = ctypes.c_char_p
        lib.lbx_strerror.argtypes = [i32]
        lib.lbx_workspace_size.restype = ctypes.c_size_t
        lib.lbx_workspace_size.argtypes = [vp]
        lib.lbx_tree_conv.restype = i32
        lib.lbx_tree_conv.argtypes = [vp] * 9
        lib.lbx_tree_deltanet.restype = i32
        lib.lbx_tree_deltanet.argtypes = [vp] * 11
        lib.lbx_tree_persist.restype = i32
        lib.lbx_tree_persist.argtypes = [vp] * 10
        lib.lbx_verify_step.restype = i32
        lib.lbx_verify_step.argtypes = [vp] * 11 + [vp, ctypes.c_size_t, vp, vp]
        lib.lbx_verify_step_noalloc.restype = i32
        lib.lbx_verify_step_noalloc.argtypes = [vp] * 13
        lib.lbx_accept_workspace_size.restype = ctypes.c_size_t
        lib.lbx_accept_workspace_size.argtypes = [i32, i32, i32]
        lib.lbx_accept_walk.restype = i32
        lib.lbx_accept_walk.argtypes = [i32, i32, i32] + [vp] * 6 + [vp, ctypes.c_size_t, vp, vp]
        lib.lbx_ddtree_build.restype = i32
        lib.lbx_ddtree_build.argtypes = [i32, i32, i32, i32] + [vp] * 9
        lib.lbx_attn_workspace_size.restype = ctypes.c_size_t
        lib.lbx_attn_workspace_size.argtypes = [i32] * 7
        lib.lbx_tree_attention.restype = i32
        lib.lbx_tree_attention.argtypes = ([i32] * 7 + [ctypes.c_float] + [vp] * 8
                                           + [vp, ctypes.c_size_t, vp, vp])
        lib.lbx_cache_attn_workspace_size.restype = ctypes.c_size_t
        lib.lbx_cache_attn_workspace_size.argtypes = [vp]
        lib.lbx_window_attention.restype = i32
        lib.lbx_window_attention.argtypes = [vp] * 10 + [vp, ctypes.c_size_t, vp, vp]
        lib.lbx_prefix_attention.restype = i32
        lib.lbx_prefix_attention.argtypes = [vp] * 12 + [vp, ctypes.c_size_t, vp, vp]
        lib.lbx_attention_mass.restype = i32
        lib.lbx_attention_mass.argtypes = [vp] * 12
        lib.lbx_cache_evict.restype = i32
        lib.lbx_cache_evict.argtypes = [vp, i32, i32] + [vp] * 15
        lib.lbx_page_tables.restype = i32
        lib.lbx_page_tables.argtypes = [vp] * 14
        lib.lbx_qk_norm_rope.restype = i32
        lib.lbx_qk_norm_rope.argtypes = [vp] * 13
        lib.lbx_paged_workspace_size.restype = ctypes.c_size_t
        lib.lbx_paged_workspace_size.argtypes = [vp]
        lib.lbx_paged_attention.restype = i32
        lib.lbx_paged_attention.argtypes = [vp] * 10 + [vp, ctypes.c_size_t, vp, vp]
        lib.lbx_page_commit.restype = i32
        lib.lbx_page_commit.argtypes = [vp] * 11
        _lib = lib
    return _lib


def strerror(rc: int) -> str:
    return load().lbx_strerror(rc).decode()


def make_cfg(L, Bq, N, Hk, Hv, d, K=4, n_slots=None, l2_eps=1e-6, q_scale=1.0,
             mode=LBX_MODE_AUTO) -> lbx_cfg:
    return lbx_cfg(L=L, Bq=Bq, N=N, Hk=Hk, Hv=Hv, d=d, K=K,
                   n_slots=Bq if n_slots is None else n_slots, l2_eps=l2_eps, q_scale=q_scale,
                   mode=mode)


def cfg_of(w, mode=LBX_MODE_AUTO) -> lbx_cfg:
    """Config from an inputs.Workload."""
    return make_cfg(w.L, w.Bq, w.N, w.Hk, w.Hv, w.d, w.K, w.n_slots, w.l2_eps, w.q_scale, mode)


_BF16_OK = (torch.bfloat16, torch.int16, getattr(torch, "uint16", torch.int16))


def _ptr(t: Optional[torch.Tensor], dtypes=None, name="") -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    return t.data_ptr()


def _bf(t, name):
    return _ptr(t, _BF16_OK, name)


def _f32(t, name):
    return _ptr(t, (torch.float32,), name)


def _i32(t, name):
    return _ptr(t, (torch.int32,), name)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, rc: int):
    if rc != LBX_OK:
        raise LbxError(fn, rc)


def lbx_workspace_size(cfg: lbx_cfg) -> int:
    return int(load().lbx_workspace_size(ctypes.byref(cfg)))


def lbx_tree_conv(cfg, x, conv_w, conv_cache, parent, slot, qkv_out, d_status=None, stream=None):
    _check("lbx_tree_conv", load().lbx_tree_conv(
        ctypes.byref(cfg), _bf(x, "x"), _bf(conv_w, "conv_w"), _f32(conv_cache, "conv_cache"),
        _i32(parent, "parent"), _i32(slot, "slot"), _f32(qkv_out, "qkv_out"),
        _i32(d_status, "d_status"), _stream(stream)))


def lbx_tree_deltanet(cfg, qkv, a, b, state, parent, slot, o, node_states=None, d_status=None,
                      stream=None):
    _check("lbx_tree_deltanet", load().lbx_tree_deltanet(
        ctypes.byref(cfg), _f32(qkv, "qkv"), _bf(a, "a"), _bf(b, "b"), _f32(state, "state"),
        _i32(parent, "parent"), _i32(slot, "slot"), _f32(o, "o"),
        _f32(node_states, "node_states"), _i32(d_status, "d_status"), _stream(stream)))


def lbx_tree_persist(cfg, x, node_states, parent, slot, accepted, state, conv_cache,
                     d_status=None, stream=None):
    _check("lbx_tree_persist", load().lbx_tree_persist(
        ctypes.byref(cfg), _bf(x, "x"), _f32(node_states, "node_states"), _i32(parent, "parent"),
        _i32(slot, "slot"), _i32(accepted, "accepted"), _f32(state, "state"),
        _f32(conv_cache, "conv_cache"), _i32(d_status, "d_status"), _stream(stream)))


def lbx_verify_step(cfg, x, conv_w, a, b, parent, slot, accepted, state, conv_cache, o,
                    workspace, d_status=None, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("lbx_verify_step", load().lbx_verify_step(
        ctypes.byref(cfg), _bf(x, "x"), _bf(conv_w, "conv_w"), _bf(a, "a"), _bf(b, "b"),
        _i32(parent, "parent"), _i32(slot, "slot"), _i32(accepted, "accepted"),
        _f32(state, "state"), _f32(conv_cache, "conv_cache"), _f32(o, "o"),
        _ptr(workspace, None, "workspace"), ws_bytes, _i32(d_status, "d_status"),
        _stream(stream)))


def lbx_verify_step_noalloc(cfg, x, conv_w, a, b, parent, slot, accepted, state, conv_cache, o,
                            d_status=None, stream=None):
    """lbx_verify_step for callers that cannot allocate: the arrival counters
    live in a fixed array inside the library (see include/lbx.h)."""
    _check("lbx_verify_step_noalloc", load().lbx_verify_step_noalloc(
        ctypes.byref(cfg), _bf(x, "x"), _bf(conv_w, "conv_w"), _bf(a, "a"), _bf(b, "b"),
        _i32(parent, "parent"), _i32(slot, "slot"), _i32(accepted, "accepted"),
        _f32(state, "state"), _f32(conv_cache, "conv_cache"), _f32(o, "o"),
        _i32(d_status, "d_status"), _stream(stream)))


def new_workspace(cfg: lbx_cfg, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of lbx_workspace_size(cfg) bytes."""
    n = lbx_workspace_size(cfg)
    if n == 0:
        raise LbxError("lbx_workspace_size", LBX_EINVAL)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lbx_accept_workspace_size(Bq: int, N: int, V: int) -> int:
    return int(load().lbx_accept_workspace_size(Bq, N, V))


def new_accept_workspace(Bq: int, N: int, V: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of lbx_accept_workspace_size(Bq, N, V) bytes."""
    n = lbx_accept_workspace_size(Bq, N, V)
    if n == 0:
        raise LbxError("lbx_accept_workspace_size", LBX_EINVAL)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lbx_accept_walk(logits, draft, parent, accepted_out, next_out, workspace, argmax_out=None,
                    d_status=None, stream=None):
    """Verify argmax and greedy acceptance walk; logits float32 [Bq][N][V]."""
    Bq, N, V = logits.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("lbx_accept_walk", load().lbx_accept_walk(
        Bq, N, V, _f32(logits, "logits"), _i32(draft, "draft"), _i32(parent, "parent"),
        _i32(argmax_out, "argmax_out"), _i32(accepted_out, "accepted_out"),
        _i32(next_out, "next_out"), _ptr(workspace, None, "workspace"), ws_bytes,
        _i32(d_status, "d_status"), _stream(stream)))


def lbx_ddtree_build(logp, tok, root_tok, B, parent_out, token_out, n_nodes_out,
                     depth_out=None, score_out=None, stream=None):
    """DDTree construction of budget B from logp float32 [Bq][D][K] and tok
    int32 [Bq][D][K]."""
    Bq, D, K = logp.shape
    _check("lbx_ddtree_build", load().lbx_ddtree_build(
        Bq, D, K, int(B), _f32(logp, "logp"), _i32(tok, "tok"), _i32(root_tok, "root_tok"),
        _i32(parent_out, "parent_out"), _i32(token_out, "token_out"),
        _i32(depth_out, "depth_out"), _f32(score_out, "score_out"),
        _i32(n_nodes_out, "n_nodes_out"), _stream(stream)))


def lbx_attn_workspace_size(L: int, Bq: int, N: int, Hq: int, Hkv: int, dh: int, T: int) -> int:
    return int(load().lbx_attn_workspace_size(L, Bq, N, Hq, Hkv, dh, T))


def new_attn_workspace(L, Bq, N, Hq, Hkv, dh, T, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of lbx_attn_workspace_size(...) bytes."""
    n = lbx_attn_workspace_size(L, Bq, N, Hq, Hkv, dh, T)
    if n == 0:
        raise LbxError("lbx_attn_workspace_size", LBX_EINVAL)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lbx_tree_attention(scale, ctx_len, parent, q, k_cache, v_cache, k_tree, v_tree, o, workspace,
                       d_status=None, stream=None):
    """Tree-masked attention of the full-attention layers: q bf16
    [L][Bq][N][Hq][dh], k_cache / v_cache [L][Bq][T][Hkv][dh], k_tree / v_tree
    [L][Bq][N][Hkv][dh], o float32 like q; shapes are read from the tensors."""
    L, Bq, N, Hq, dh = q.shape
    T, Hkv = k_cache.shape[2], k_cache.shape[3]
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("lbx_tree_attention", load().lbx_tree_attention(
        L, Bq, N, Hq, Hkv, dh, T, float(scale), _i32(ctx_len, "ctx_len"), _i32(parent, "parent"),
        _bf(q, "q"), _bf(k_cache, "k_cache") if T > 0 else None,
        _bf(v_cache, "v_cache") if T > 0 else None, _bf(k_tree, "k_tree"), _bf(v_tree, "v_tree"),
        _f32(o, "o"), _ptr(workspace, None, "workspace"), ws_bytes, _i32(d_status, "d_status"),
        _stream(stream)))


def make_attn_cfg(L, Bq, N, Hq, Hkv, dh, T, P=0, window=0, n_sink=0, dtype=LBX_BF16,
                  scale=None) -> lbx_attn_cfg:
    """Config of the bounded cache's operators; scale defaults to 1/sqrt(dh)."""
    return lbx_attn_cfg(L=L, Bq=Bq, N=N, Hq=Hq, Hkv=Hkv, dh=dh, T=T, P=P, window=window,
                        n_sink=n_sink, dtype=dtype, scale=dh ** -0.5 if scale is None else scale)


_ELEM = {LBX_BF16: torch.bfloat16, LBX_F16: torch.float16}


def _refuse(t, shape, dtype, name):
    """What _at refused, said in _ptr's words."""
    ok = _BF16_OK if dtype is torch.bfloat16 else (dtype,)
    p = _ptr(t, ok, name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    return p


def _at(t, shape, dtype, name):
    """The address of a contiguous CUDA tensor of this shape and type (the calls
    below check a dozen of them, which for a small call costs as much as the
    kernel: one line for the ordinary case)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda
            and t.is_contiguous()):
        return t.data_ptr()
    return _refuse(t, shape, dtype, name)


def _public_raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The current stream's handle without a Stream object around it, which costs 2 us per
# call, a fifth of the smallest calls; torch does not promise this name.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)


def _stream_of(t, stream):
    """The given stream, or the current one of the tensor's device."""
    if stream is None:
        return _raw_stream(t.get_device())
    return _stream(stream)


def lbx_cache_attn_workspace_size(cfg: lbx_attn_cfg) -> int:
    return int(load().lbx_cache_attn_workspace_size(ctypes.byref(cfg)))


def new_cache_attn_workspace(cfg: lbx_attn_cfg, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of lbx_cache_attn_workspace_size(cfg) bytes."""
    n = lbx_cache_attn_workspace_size(cfg)
    if n == 0:
        raise LbxError("lbx_cache_attn_workspace_size", LBX_EINVAL)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _attention_arrays(cfg, ctx_len, parent, q, prefix, k_cache, v_cache, k_tree, v_tree, o, lse):
    """Addresses of the attention calls' arrays in the C order."""
    L, Bq, N, Hq, Hkv, dh, T = cfg.L, cfg.Bq, cfg.N, cfg.Hq, cfg.Hkv, cfg.dh, cfg.T
    el, i32 = _ELEM.get(cfg.dtype, torch.bfloat16), torch.int32
    qs, cs, ts = (L, Bq, N, Hq, dh), (L, Bq, T, Hkv, dh), (L, Bq, N, Hkv, dh)
    return (_at(ctx_len, (Bq,), i32, "ctx_len"), _at(parent, (Bq, N), i32, "parent"),
            _at(q, qs, el, "q"), *prefix, _at(k_cache, cs, el, "k_cache"),
            _at(v_cache, cs, el, "v_cache"), _at(k_tree, ts, el, "k_tree"),
            _at(v_tree, ts, el, "v_tree"), _at(o, qs, el, "o"),
            None if lse is None else _at(lse, (L, Bq, N, Hq), torch.float32, "lse"))


def lbx_window_attention(cfg, ctx_len, parent, q, k_cache, v_cache, k_tree, v_tree, o, workspace,
                         lse=None, d_status=None, stream=None):
    """Tree attention with a sliding window and visible first positions."""
    _check("lbx_window_attention", load().lbx_window_attention(
        ctypes.byref(cfg), *_attention_arrays(cfg, ctx_len, parent, q, (), k_cache, v_cache,
                                              k_tree, v_tree, o, lse),
        _ptr(workspace, None, "workspace"), workspace.nbytes, _i32(d_status, "d_status"),
        _stream_of(q, stream)))


def lbx_prefix_attention(cfg, ctx_len, parent, q, k_prefix, v_prefix, k_cache, v_cache, k_tree,
                         v_tree, o, workspace, lse=None, d_status=None, stream=None):
    """Attention of a batch over one shared prefix, its own caches and trees."""
    el, ps = _ELEM.get(cfg.dtype, torch.bfloat16), (cfg.L, cfg.P, cfg.Hkv, cfg.dh)
    prefix = _at(k_prefix, ps, el, "k_prefix"), _at(v_prefix, ps, el, "v_prefix")
    _check("lbx_prefix_attention", load().lbx_prefix_attention(
        ctypes.byref(cfg), *_attention_arrays(cfg, ctx_len, parent, q, prefix, k_cache, v_cache,
                                              k_tree, v_tree, o, lse),
        _ptr(workspace, None, "workspace"), workspace.nbytes, _i32(d_status, "d_status"),
        _stream_of(q, stream)))


def lbx_attention_mass(cfg, ctx_len, parent, accepted, q, lse, k_cache, k_tree, score, score_tree,
                       d_status=None, stream=None):
    """Accumulate the accepted path's attention weights per key."""
    L, Bq, N, Hq, Hkv, dh, T = cfg.L, cfg.Bq, cfg.N, cfg.Hq, cfg.Hkv, cfg.dh, cfg.T
    el, i32, f32 = _ELEM.get(cfg.dtype, torch.bfloat16), torch.int32, torch.float32
    _check("lbx_attention_mass", load().lbx_attention_mass(
        ctypes.byref(cfg), _at(ctx_len, (Bq,), i32, "ctx_len"),
        _at(parent, (Bq, N), i32, "parent"), _at(accepted, (Bq,), i32, "accepted"),
        _at(q, (L, Bq, N, Hq, dh), el, "q"), _at(lse, (L, Bq, N, Hq), f32, "lse"),
        _at(k_cache, (L, Bq, T, Hkv, dh), el, "k_cache"),
        _at(k_tree, (L, Bq, N, Hkv, dh), el, "k_tree"), _at(score, (L, Bq, Hkv, T), f32, "score"),
        _at(score_tree, (L, Bq, Hkv, N), f32, "score_tree"), _i32(d_status, "d_status"),
        _stream_of(q, stream)))


def lbx_cache_evict(cfg, budget, n_recent, ctx_len, seen, parent, accepted, k_tree, v_tree,
                    score_tree, k_cache, v_cache, score, pos, ctx_out, seen_out, d_status=None,
                    stream=None):
    """Append the accepted path to the cache and keep its `budget` best entries."""
    L, Bq, N, Hkv, dh, T = cfg.L, cfg.Bq, cfg.N, cfg.Hkv, cfg.dh, cfg.T
    el, i32, f32 = _ELEM.get(cfg.dtype, torch.bfloat16), torch.int32, torch.float32
    cs, ts, per = (L, Bq, T, Hkv, dh), (L, Bq, N, Hkv, dh), (Bq,)
    _check("lbx_cache_evict", load().lbx_cache_evict(
        ctypes.byref(cfg), int(budget), int(n_recent), _at(ctx_len, per, i32, "ctx_len"),
        _at(seen, per, i32, "seen"), _at(parent, (Bq, N), i32, "parent"),
        _at(accepted, per, i32, "accepted"), _at(k_tree, ts, el, "k_tree"),
        _at(v_tree, ts, el, "v_tree"), _at(score_tree, (L, Bq, Hkv, N), f32, "score_tree"),
        _at(k_cache, cs, el, "k_cache"), _at(v_cache, cs, el, "v_cache"),
        _at(score, (L, Bq, Hkv, T), f32, "score"), _at(pos, (L, Bq, Hkv, T), i32, "pos"),
        _at(ctx_out, per, i32, "ctx_out"), _at(seen_out, per, i32, "seen_out"),
        _i32(d_status, "d_status"), _stream_of(score, stream)))


def make_page_cfg(L, Bq, M, Hq, Hkv, dh, page, n_pages, max_pages, dtype=LBX_BF16,
                  scale=None, weights=LBX_WEIGHTS_ROUNDED) -> lbx_page_cfg:
    """Config of the paged cache's operators; scale defaults to 1/sqrt(dh), weights says how
    the attention's softmax weights meet V (LBX_WEIGHTS_SPLIT: in two 16-bit parts)."""
    return lbx_page_cfg(L=L, Bq=Bq, M=M, Hq=Hq, Hkv=Hkv, dh=dh, page=page, n_pages=n_pages,
                        max_pages=max_pages, dtype=dtype, scale=dh ** -0.5 if scale is None else scale,
                        weights=weights)


def make_rope_cfg(sections, eps=1e-6, pairing=LBX_ROPE_HALVES) -> lbx_rope_cfg:
    """Rotation of 2 * sum(sections) dimensions; sections[a] pairs turn with axis a."""
    if len(sections) > LBX_ROPE_MAX_AXES:
        raise ValueError(f"sections: {len(sections)} axes, at most {LBX_ROPE_MAX_AXES}")
    return lbx_rope_cfg(rot=2 * sum(sections), axes=len(sections),
                        section=(ctypes.c_int * LBX_ROPE_MAX_AXES)(*sections), pairing=pairing,
                        eps=eps)


def lbx_page_tables(cfg, ctx_len, new_len, held, n_free, block_table, free_list, held_out, n_free_out,
                    start, slot, pos, d_status=None, stream=None):
    """Block tables and slot maps of a step from the requests' lengths."""
    i32, one, Bq, rows = torch.int32, (1,), cfg.Bq, (cfg.M,)
    per = (Bq,)
    rc = load().lbx_page_tables(
        ctypes.byref(cfg), _at(ctx_len, per, i32, "ctx_len"), _at(new_len, per, i32, "new_len"),
        _at(held, per, i32, "held"), _at(n_free, one, i32, "n_free"),
        _at(block_table, (Bq, cfg.max_pages), i32, "block_table"),
        _at(free_list, (cfg.n_pages,), i32, "free_list"), _at(held_out, per, i32, "held_out"),
        _at(n_free_out, one, i32, "n_free_out"), _at(start, (Bq + 1,), i32, "start"),
        _at(slot, rows, i32, "slot"), _at(pos, rows, i32, "pos"),
        None if d_status is None else _i32(d_status, "d_status"), _stream_of(slot, stream))
    if rc:
        _check("lbx_page_tables", rc)


def lbx_qk_norm_rope(cfg, rope, qkv, inv_freq, pos, slot, q_out, k_pages, v_pages, q_weight=None,
                     k_weight=None, d_status=None, stream=None):
    """Norms of queries and keys per head and their rotation; keys and values
    go to their pages."""
    el, i32, f32 = _ELEM.get(cfg.dtype, torch.bfloat16), torch.int32, torch.float32
    L, M, Hq, Hkv, dh = cfg.L, cfg.M, cfg.Hq, cfg.Hkv, cfg.dh
    pool, w = (L, cfg.n_pages, cfg.page, Hkv, dh), (L, dh)
    rc = load().lbx_qk_norm_rope(
        ctypes.byref(cfg), ctypes.byref(rope), _at(qkv, (L, M, Hq + 2 * Hkv, dh), el, "qkv"),
        None if q_weight is None else _at(q_weight, w, f32, "q_weight"),
        None if k_weight is None else _at(k_weight, w, f32, "k_weight"),
        None if inv_freq is None else _at(inv_freq, (rope.rot // 2,), f32, "inv_freq"),
        _at(pos, (rope.axes, M), i32, "pos"), _at(slot, (M,), i32, "slot"),
        _at(q_out, (L, M, Hq, dh), el, "q_out"), _at(k_pages, pool, el, "k_pages"),
        _at(v_pages, pool, el, "v_pages"), None if d_status is None else _i32(d_status, "d_status"),
        _stream_of(qkv, stream))
    if rc:
        _check("lbx_qk_norm_rope", rc)


def lbx_paged_workspace_size(cfg: lbx_page_cfg) -> int:
    return int(load().lbx_paged_workspace_size(ctypes.byref(cfg)))


def new_paged_workspace(cfg: lbx_page_cfg, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of lbx_paged_workspace_size(cfg) bytes."""
    n = lbx_paged_workspace_size(cfg)
    if n == 0:
        raise LbxError("lbx_paged_workspace_size", LBX_EINVAL)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def lbx_paged_attention(cfg, start, ctx_len, block_table, q, k_pages, v_pages, o, workspace,
                        parent=None, lse=None, d_status=None, stream=None):
    """Attention of each request's new tokens (a chunk, a tree, one token) over its pages."""
    el, i32 = _ELEM.get(cfg.dtype, torch.bfloat16), torch.int32
    L, Bq, M, Hq, dh = cfg.L, cfg.Bq, cfg.M, cfg.Hq, cfg.dh
    qs, pool = (L, M, Hq, dh), (L, cfg.n_pages, cfg.page, cfg.Hkv, dh)
    rc = load().lbx_paged_attention(
        ctypes.byref(cfg), _at(start, (Bq + 1,), i32, "start"), _at(ctx_len, (Bq,), i32, "ctx_len"),
        _at(block_table, (Bq, cfg.max_pages), i32, "block_table"),
        None if parent is None else _at(parent, (M,), i32, "parent"), _at(q, qs, el, "q"),
        _at(k_pages, pool, el, "k_pages"), _at(v_pages, pool, el, "v_pages"), _at(o, qs, el, "o"),
        None if lse is None else _at(lse, (L, M, Hq), torch.float32, "lse"),
        _ptr(workspace, None, "workspace"), workspace.nbytes,
        None if d_status is None else _i32(d_status, "d_status"), _stream_of(q, stream))
    if rc:
        _check("lbx_paged_attention", rc)


def lbx_page_commit(cfg, start, ctx_len, block_table, parent, accepted, k_pages, v_pages, ctx_out,
                    d_status=None, stream=None):
    """Move the accepted path's keys and values to the positions behind the context."""
    el, i32, Bq = _ELEM.get(cfg.dtype, torch.bfloat16), torch.int32, cfg.Bq
    per, pool = (Bq,), (cfg.L, cfg.n_pages, cfg.page, cfg.Hkv, cfg.dh)
    rc = load().lbx_page_commit(
        ctypes.byref(cfg), _at(start, (Bq + 1,), i32, "start"), _at(ctx_len, per, i32, "ctx_len"),
        _at(block_table, (Bq, cfg.max_pages), i32, "block_table"),
        _at(parent, (cfg.M,), i32, "parent"), _at(accepted, per, i32, "accepted"),
        _at(k_pages, pool, el, "k_pages"), _at(v_pages, pool, el, "v_pages"),
        _at(ctx_out, per, i32, "ctx_out"), None if d_status is None else _i32(d_status, "d_status"),
        _stream_of(k_pages, stream))
    if rc:
        _check("lbx_page_commit", rc)
