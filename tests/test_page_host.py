"""Host-side rules of the paged cache's operators, through the built library: bad
calls are refused before any launch (no GPU needed; nothing is read)."""
import ctypes

import pytest

from tree_verify_linear_gb300 import lbx


@pytest.fixture(scope="module")
def lib():
    from tree_verify_linear_gb300 import build
    build.build()
    return lbx.load()


def cfg(**kw):
    base = dict(L=2, Bq=4, M=32, Hq=8, Hkv=2, dh=64, page=16, n_pages=10, max_pages=5)
    return lbx.make_page_cfg(**{**base, **kw})


def apart(n):
    """n addresses far from each other."""
    return [(i + 1) << 28 for i in range(n)]


def call(lib, op, c, args=None, rope=None, ws=1 << 40):
    by = ctypes.byref(c)
    if op == "tables":
        return lib.lbx_page_tables(by, *(args or apart(11)), None, None)
    if op == "rope":
        return lib.lbx_qk_norm_rope(by, ctypes.byref(rope or lbx.make_rope_cfg([8])), *(args or apart(9)),
                                    None, None)
    if op == "attention":
        return lib.lbx_paged_attention(by, *(args or apart(10)), ws, None, None)
    return lib.lbx_page_commit(by, *(args or apart(8)), None, None)


BAD = [dict(L=0), dict(Bq=0), dict(Bq=2049), dict(M=0), dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(dh=96),
       dict(page=0), dict(page=48), dict(page=512), dict(page=8), dict(n_pages=0), dict(max_pages=0),
       dict(dtype=2), dict(dtype=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
       dict(scale=float("inf")), dict(L=2 ** 16, M=2 ** 16), dict(Hq=2 ** 12, Hkv=2 ** 12, M=2 ** 20),
       dict(n_pages=2 ** 27), dict(L=2 ** 20, n_pages=2 ** 10), dict(max_pages=2 ** 27),
       dict(Hkv=2 ** 24, Hq=2 ** 24, M=1)]


@pytest.mark.parametrize("kw", BAD, ids=str)
@pytest.mark.parametrize("op", ["tables", "rope", "attention", "commit"])
def test_bad_configs_are_refused(lib, op, kw):
    assert call(lib, op, cfg(**kw)) == lbx.LBX_EINVAL
    assert lbx.lbx_paged_workspace_size(cfg(**kw)) == 0


def test_a_missing_config_is_refused(lib):
    assert lib.lbx_page_tables(None, *apart(11), None, None) == lbx.LBX_EINVAL
    assert lib.lbx_qk_norm_rope(None, None, *apart(9), None, None) == lbx.LBX_EINVAL
    assert lib.lbx_qk_norm_rope(ctypes.byref(cfg()), None, *apart(9), None, None) == lbx.LBX_EINVAL
    assert lib.lbx_paged_attention(None, *apart(10), 1 << 40, None, None) == lbx.LBX_EINVAL
    assert lib.lbx_page_commit(None, *apart(8), None, None) == lbx.LBX_EINVAL
    assert lib.lbx_paged_workspace_size(None) == 0


# (operator, argument): those that may be NULL and those whose alignment is 4
MAY_BE_NULL = {("rope", 1), ("rope", 2), ("attention", 3), ("attention", 8)}
WORDS = {"tables": range(11), "rope": (3, 4, 5), "attention": (0, 1, 2, 3, 8), "commit": (0, 1, 2, 3, 4, 7)}
COUNT = {"tables": 11, "rope": 9, "attention": 10, "commit": 8}


@pytest.mark.parametrize("op,i", [(op, i) for op, n in COUNT.items() for i in range(n)])
def test_null_and_misaligned_arrays_are_refused(lib, op, i):
    for at in ([] if (op, i) in MAY_BE_NULL else [None]) + [2] + ([] if i in WORDS[op] else [8]):
        args = apart(COUNT[op])
        args[i] = None if at is None else args[i] + at
        assert call(lib, op, cfg(), args) == lbx.LBX_EINVAL, at


def test_status_words_are_aligned(lib):
    by = ctypes.byref(cfg())
    assert lib.lbx_page_tables(by, *apart(11), 2, None) == lbx.LBX_EINVAL
    assert lib.lbx_qk_norm_rope(by, ctypes.byref(lbx.make_rope_cfg([8])), *apart(9), 2, None) == lbx.LBX_EINVAL
    assert lib.lbx_paged_attention(by, *apart(10), 1 << 40, 2, None) == lbx.LBX_EINVAL
    assert lib.lbx_page_commit(by, *apart(8), 2, None) == lbx.LBX_EINVAL


# ctx_len, new_len, held, n_free are 0..3; held_out, n_free_out, start, slot, pos 6..10
@pytest.mark.parametrize("out", [4, 5, 6, 7, 8, 9, 10])
@pytest.mark.parametrize("on", [0, 1, 2, 3])
def test_tables_refuse_outputs_over_inputs(lib, out, on):
    size = 4 if on == 3 else 16
    for at in (0, size - 4):
        args = apart(11)
        args[out] = args[on] + at
        assert call(lib, "tables", cfg(), args) == lbx.LBX_EINVAL, at


@pytest.mark.parametrize("a,b", [(6, 7), (6, 8), (9, 10), (4, 5), (5, 9)])
def test_tables_refuse_outputs_over_each_other(lib, a, b):
    args = apart(11)
    args[b] = args[a]
    assert call(lib, "tables", cfg(), args) == lbx.LBX_EINVAL


@pytest.mark.parametrize("on,size", [(0, 20), (1, 16), (2, 80), (3, 128), (4, 16)])
def test_commit_refuses_lengths_over_its_inputs(lib, on, size):
    for at in (-12, 0, size - 4):
        args = apart(8)
        args[7] = args[on] + at
        assert call(lib, "commit", cfg(), args) == lbx.LBX_EINVAL, at


@pytest.mark.parametrize("op", ["tables", "rope", "attention", "commit"])
@pytest.mark.parametrize("dh", [64, 128, 256])
def test_rows_of_a_gigabyte_are_refused(lib, op, dh):
    assert call(lib, op, cfg(L=1, M=1, Hq=2 ** 29 // dh, Hkv=2 ** 22 // dh, dh=dh)) == lbx.LBX_EINVAL


# 2 layers of 32 rows: q has 8 heads of 64, qkv 12; lse a word per head
@pytest.mark.parametrize("at", [0, 2 * 32 * 12 * 128 - 16, 16 - 2 * 32 * 8 * 128])
def test_rotation_refuses_queries_over_its_input(lib, at):
    args = apart(9)
    args[6] = args[0] + at
    assert call(lib, "rope", cfg(), args) == lbx.LBX_EINVAL


# q is 4, o 7, lse 8, the workspace 9
@pytest.mark.parametrize("out,on,size,own", [(7, 4, 65536, 65536), (8, 4, 65536, 2048), (8, 7, 65536, 2048),
                                             (9, 4, 65536, 4096), (9, 7, 65536, 4096), (9, 8, 2048, 4096)])
def test_attention_refuses_outputs_over_queries_and_each_other(lib, out, on, size, own):
    for at in (0, size - 16, 16 - own):
        args = apart(10)
        args[out] = args[on] + at
        assert call(lib, "attention", cfg(), args) == lbx.LBX_EINVAL, at


BAD_ROPE = [dict(rot=-2), dict(rot=3), dict(rot=66), dict(axes=0), dict(axes=5), dict(pairing=2),
            dict(pairing=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rot=18)]


@pytest.mark.parametrize("kw", BAD_ROPE, ids=str)
def test_bad_rotations_are_refused(lib, kw):
    r = lbx.make_rope_cfg([8])
    for k, v in kw.items():
        setattr(r, k, v)
    assert call(lib, "rope", cfg(), rope=r) == lbx.LBX_EINVAL


@pytest.mark.parametrize("axes,section", [(1, (4, 4, 0, 0)), (2, (-1, 9, 0, 0)), (3, (2, 2, 2, 2)),
                                          (4, (2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30))])
def test_bad_sections_are_refused(lib, axes, section):
    r = lbx.make_rope_cfg([8])
    r.axes = axes
    for i, n in enumerate(section):
        r.section[i] = n
    assert call(lib, "rope", cfg(), rope=r) == lbx.LBX_EINVAL


def test_too_many_axes_are_refused_by_the_binding():
    with pytest.raises(ValueError):
        lbx.make_rope_cfg([1] * 5)


def test_wide_groups_and_short_workspaces_are_refused(lib):
    wide = cfg(Hq=129, Hkv=1)
    assert lbx.lbx_paged_workspace_size(wide) == 0
    assert call(lib, "attention", wide) == lbx.LBX_EINVAL
    need = lbx.lbx_paged_workspace_size(cfg())
    assert need > 0 and call(lib, "attention", cfg(), ws=need - 1) == lbx.LBX_EINVAL
    with pytest.raises(lbx.LbxError):
        lbx.new_paged_workspace(wide, device="cpu")


def test_the_new_status_has_a_text(lib):
    assert "pages" in lbx.strerror(lbx.LBX_EPAGES)
