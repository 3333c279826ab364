"""Arrays that the binding's calls refuse before the library sees an address (no GPU needed)."""
import pytest
import torch

from tree_verify_linear_gb300 import lbx


class Like:
    """Looks like a contiguous CUDA tensor, and is none."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, True

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("an address was asked for")


@pytest.mark.parametrize("make", [lambda shape, dtype: Like(shape, dtype),
                                  lambda shape, dtype: torch.zeros(shape, dtype=dtype),
                                  lambda shape, dtype: [0]], ids=["look_alike", "host_tensor", "list"])
def test_only_cuda_tensors_have_addresses(make):
    bf16, i32 = torch.bfloat16, torch.int32
    for shape, dtype in (((2, 3), i32), ((1, 4, 2, 64), bf16)):
        with pytest.raises(TypeError, match="expected a CUDA tensor"):
            lbx._at(make(shape, dtype), shape, dtype, "x")
    cfg = lbx.make_page_cfg(1, 1, 1, 2, 1, 64, 16, 4, 4)
    per, rows = make((1,), i32), make((1,), i32)
    with pytest.raises(TypeError, match="expected a CUDA tensor"):
        lbx.lbx_page_tables(cfg, per, per, per, per, make((1, 4), i32), make((4,), i32), per, per,
                            make((2,), i32), rows, rows, stream=0)
