"""Where each CTA of lbx_paged_attention finds its work, on the device."""
import os
import subprocess

import pytest

from tree_verify_linear_gb300 import build

pytestmark = pytest.mark.gpu


def test_ranges_begin_where_the_list_says(tmp_path):
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "check")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-I", build.INCLUDE,
                    "-I", build.CSRC, "-o", exe, os.path.join(here, "page_begin_check.cu")], check=True,
                   capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
