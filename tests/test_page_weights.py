"""The choice of how weights meet V, checked on the host (no GPU needed)."""
import pytest

from test_page_host import call, cfg, lib  # noqa: F401
from tree_verify_linear_gb300 import lbx


@pytest.mark.parametrize("op", ["tables", "rope", "attention", "commit"])
@pytest.mark.parametrize("weights", [-1, 2])
def test_other_choices_are_refused(lib, op, weights):  # noqa: F811
    assert call(lib, op, cfg(weights=weights)) == lbx.LBX_EINVAL
    assert lbx.lbx_paged_workspace_size(cfg(weights=weights)) == 0


def test_both_choices_take_one_workspace(lib):  # noqa: F811
    assert cfg().weights == lbx.LBX_WEIGHTS_ROUNDED
    assert lbx.lbx_paged_workspace_size(cfg(weights=lbx.LBX_WEIGHTS_SPLIT)) == lbx.lbx_paged_workspace_size(cfg())
