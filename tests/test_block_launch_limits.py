"""The block operators' launches at the largest sizes that their argument checks let through, on
the CPU: the HIP sources compiled for the host only and linked with the stub runtime."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "selective_state_space_79_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
CLANG = "/opt/rocm/lib/llvm/bin/clang++"


def _run(cmd, timeout=300):
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=timeout)
    assert r.returncode == 0, r.stderr[-3000:]
    return r


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not installed")
def test_launches_stay_within_the_grid_limits(tmp_path):
    inc = ["-I", os.path.join(ROOT, "include")]
    objs, procs = [], []
    for name in ("linattn_fwd", "linattn_bwd", "norms"):
        objs.append(str(tmp_path / f"{name}.o"))
        procs.append(subprocess.Popen([HIPCC, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17", "-fPIC", *inc, "-c",
                                       "-o", objs[-1], os.path.join(CSRC, f"{name}.hip")], stdout=subprocess.PIPE,
                                      stderr=subprocess.PIPE, text=True))
    for pr in procs:
        _, err = pr.communicate(timeout=600)
        assert pr.returncode == 0, err[-3000:]
    syms = set()
    for obj in objs:
        syms |= set(re.findall(r"\b(__hip_fatbin_[0-9a-f]+)\b", _run(["nm", "-u", obj]).stdout))
    (tmp_path / "fatbin_symbols.inc").write_text("".join(f"SSM_STUB_FATBIN({s})\n" for s in sorted(syms)))
    exe = str(tmp_path / "launch_limit_checks")
    _run([CLANG, "-O1", "-std=c++17", *inc, "-I", "/opt/rocm/include", "-I", str(tmp_path), "-D__HIP_PLATFORM_AMD__", "-o", exe,
          os.path.join(HERE, "launch_limit_checks.cpp"), os.path.join(HERE, "hip_stub.cpp"), *objs, "-lpthread"], timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]
