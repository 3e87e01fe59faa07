"""Offsets that the block operators' kernels form, checked on the CPU over the sizes that the
entry points allow (the header compiled for the host)."""
import os
import subprocess

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="ROCm compilers not installed")
def test_outputs_past_the_last_column_are_dropped(tmp_path):
    """Rows of all heads reach 33 MB (the gradients' float32 rows per head): a store of a column
    that the head does not have must stay past the chunk's window, also against time."""
    exe = str(tmp_path / "store_rows_checks")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "selective_state_space_79_amd", "csrc"), "-o", exe,
                    "-x", "hip", os.path.join(HERE, "store_rows_checks.cpp")], check=True, timeout=300, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
