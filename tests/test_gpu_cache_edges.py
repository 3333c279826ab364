"""GPU tests of the bounded cache's operators at their edges: full windows,
shared workspaces, calls side by side, NaN, the longest windows."""
import numpy as np
import pytest
import torch

import cache_ref as R
from test_gpu_cache import built, check_attention, run_attention, run_mass  # noqa: F401 (built: a fixture)

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
