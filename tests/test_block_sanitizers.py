"""The block operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer on the
CPU, as test_host_sanitizers.py does for the scan: the HIP sources compiled for the host only
and linked with the stub runtime of tests/sanitize/hip_stub.cpp."""
import os
import re
import subprocess

import pytest

from test_host_sanitizers import CLANG, CSRC, ENV, HERE, HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not installed")
def test_block_host_code_under_sanitizers(tmp_path):
    host = ["--offload-arch=gfx950", "--cuda-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-I",
            os.path.join(ROOT, "include")]
    for flag in SAN:
        host += ["-Xarch_host", flag]
    objs, procs = [], []
    for name in ("linattn_fwd", "linattn_bwd", "norms"):
        obj = str(tmp_path / f"{name}.o")
        objs.append(obj)
        procs.append(subprocess.Popen([HIPCC, *host, "-c", "-o", obj, os.path.join(CSRC, f"{name}.hip")],
                                      stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True))
    for pr in procs:
        _, err = pr.communicate(timeout=600)
        assert pr.returncode == 0, err[-3000:]
    syms = set()
    for obj in objs:
        syms |= set(re.findall(r"\b(__hip_fatbin_[0-9a-f]+)\b", _run(["nm", "-u", obj]).stdout))
    (tmp_path / "fatbin_symbols.inc").write_text("".join(f"SSM_STUB_FATBIN({s})\n" for s in sorted(syms)))
    exe = str(tmp_path / "block_host_checks")
    _run([CLANG, "-O1", "-g", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
          "-I", str(tmp_path), "-D__HIP_PLATFORM_AMD__", "-o", exe, os.path.join(HERE, "block_host_checks.cpp"),
          os.path.join(HERE, "hip_stub.cpp"), *objs, "-lpthread"], timeout=600)
    r = _run([exe], env=ENV, timeout=600)
    print(r.stdout)
    assert "0 failed" in r.stdout
