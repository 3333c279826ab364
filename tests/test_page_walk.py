"""How lbx_paged_attention shares out its work, checked on the host (no GPU needed)."""
import os
import subprocess

from tree_verify_linear_gb300 import build


def test_ranges_cover_every_block_once(tmp_path):
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "check")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
                    "-o", exe, os.path.join(here, "page_walk_check.cu")], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
