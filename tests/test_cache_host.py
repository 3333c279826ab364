"""Host-side rules of the bounded cache's operators, through the built library
(no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from tree_verify_linear_gb300 import build, lbx
    build.build()
    return lbx.load()


def units(n):
    return -(-n // 64)


def units_of(ctx, window, n_sink):
    """Units of 64 keys in a request's list: visible first positions before the
    window, the window, the tree."""
    w0 = max(0, ctx - window + 1) if window else 0
    return units(min(n_sink, w0)) + units(ctx - w0) + 1


def test_the_small_kernel_has_a_block_for_every_unit(lib):
    """Whatever the context length, no request has more units than the launch has
    blocks per stream, and some has as many."""
    from tree_verify_linear_gb300 import lbx
    chunks = lib._ZN3lbx5cache10few_chunksEPK12lbx_attn_cfg
    chunks.argtypes, chunks.restype = [ctypes.c_void_p], ctypes.c_int
    for T in (0, 1, 2, 63, 64, 65, 100, 127, 128, 129, 512, 1000, 1024):
        for window in sorted({0, 1, 2, 63, 64, 65, 66, 129, T // 2, T - 1, T, T + 1, 5000, 2**31 - 1}):
            for n_sink in (0, 1, 4, 64, 65, T, 2**31 - 1):
                if window < 0:
                    continue
                cfg = lbx.make_attn_cfg(1, 1, 1, 4, 1, 64, T, window=window, n_sink=n_sink)
                got = chunks(ctypes.byref(cfg))
                most = max(units_of(ctx, window, n_sink) for ctx in range(T + 1))
                assert got == most, (T, window, n_sink)


@pytest.mark.parametrize("out,on", [(o, i) for o in (11, 12) for i in (0, 1, 2, 3)] + [(11, 12)])
@pytest.mark.parametrize("at", [-60, 0, 60])
def test_eviction_refuses_outputs_over_its_inputs(lib, out, on, at):
    """Arguments 11 and 12 are ctx_out and seen_out, 0 to 3 ctx_len, seen, parent
    and accepted, 16 requests each (nothing is read: the call is refused first)."""
    from tree_verify_linear_gb300 import lbx
    cfg = lbx.make_attn_cfg(L=1, Bq=16, N=4, Hq=4, Hkv=2, dh=64, T=8)
    args = [(i + 1) << 20 for i in range(13)]
    args[out] = args[on] + at
    assert lib.lbx_cache_evict(ctypes.byref(cfg), 4, 0, *args, None, None) == lbx.LBX_EINVAL
