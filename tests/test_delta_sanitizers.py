"""The host code of the gated delta rule and of the layer norm under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU: the HIP sources compiled for the host only and linked with
the stub runtime of tests/sanitize/hip_stub.cpp, which checks every launch."""
import os
import re
import subprocess

import pytest

from test_host_sanitizers import CLANG, CSRC, ENV, HERE, HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not installed")
def test_delta_host_code_under_sanitizers(tmp_path):
    host = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-I",
            os.path.join(ROOT, "include")]
    for flag in SAN:
        host += ["-Xarch_host", flag]
    objs, procs = [], []
    for name in ("delta_fwd", "delta_bwd", "norms"):
        objs.append(str(tmp_path / f"{name}.o"))
        procs.append(subprocess.Popen([HIPCC, *host, "-c", "-o", objs[-1], os.path.join(CSRC, f"{name}.hip")],
                                      stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
    for pr in procs:
        _, err = pr.communicate(timeout=600)
        assert pr.returncode == 0, err[-3000:]
    syms = set()
    for obj in objs:
        syms |= set(re.findall(r"\b(__hip_fatbin_[0-9a-f]+)\b", _run(["nm", "-u", obj]).stdout))
    (tmp_path / "fatbin_symbols.inc").write_text("".join(f"SSM_STUB_FATBIN({s})\n" for s in sorted(syms)))
    exe = str(tmp_path / "delta_host_checks")
    _run([CLANG, "-O1", "-g", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
          "-I", str(tmp_path), "-D__HIP_PLATFORM_AMD__", "-o", exe, os.path.join(HERE, "delta_host_checks.cpp"),
          os.path.join(HERE, "hip_stub.cpp"), *objs, "-lpthread"], timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=ENV)
    assert r.returncode == 0, r.stdout + r.stderr[:3000]
