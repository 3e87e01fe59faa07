"""The sizes that the gated delta rule takes and refuses, on the CPU (the HIP sources compiled for
the host only and linked with the stub runtime, which checks every launch), and calls of more
sequences than an earlier limit let through, on the GPU."""
import os
import re
import subprocess

import pytest

from test_block_launch_limits import CLANG, CSRC, HERE, HIPCC, ROOT, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm compilers not installed")
def test_sizes_within_the_limits_are_taken(tmp_path):
    inc = ["-I", os.path.join(ROOT, "include")]
    objs, procs = [], []
    for name in ("delta_fwd", "delta_bwd"):
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
    exe = str(tmp_path / "delta_limit_checks")
    _run([CLANG, "-O1", "-std=c++17", *inc, "-I", "/opt/rocm/include", "-I", str(tmp_path), "-D__HIP_PLATFORM_AMD__", "-o", exe,
          os.path.join(HERE, "delta_limit_checks.cpp"), os.path.join(HERE, "hip_stub.cpp"), *objs, "-lpthread"], timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]


@pytest.mark.gpu
def test_forward_of_very_many_short_sequences():
    """40000 sequences of one token each and 32 heads of 128 x 128, 2.6 million workgroups.  From zeros
    o = scale beta (q . k) v: a product of 128 terms, each rounded by 2^-24 of |q| |k| <= 1 at most, and
    four more roundings, so within 2^-16 |beta v| scale, and 2^-8 of the value in bf16."""
    import torch
    import selective_state_space_79_amd as ssm

    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    print("\n[gpu-case] delta 40000 sequences of one token", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    n, H, d = 40000, 32, 128
    q, k = (torch.nn.functional.normalize(torch.randn(n, 1, d, generator=gen, device="cuda"), dim=-1).bfloat16() for _ in range(2))
    v = torch.randn(n, H, d, generator=gen, device="cuda").bfloat16()
    g, beta = torch.zeros(n, H, device="cuda"), torch.rand(n, H, generator=gen, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    o = ssm.delta_fwd(q, k, v, g, beta, scale=0.5, cu_seqlens=cu)
    torch.cuda.synchronize()
    u = 0.5 * beta[..., None].double() * v.double()
    want = (q.double() * k.double()).sum(-1, keepdim=True) * u
    assert ((o.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * u.abs()).all()


@pytest.mark.gpu
def test_gradients_of_very_many_short_sequences():
    """40000 float32 sequences of one token each and 64 heads of 16 x 16, 5.1 million workgroups of the
    two walks.  From zeros u = beta v, o = scale (q . k) u, so with c = scale (q . k), e = scale (do . u):
    dv = beta c do, dbeta = c (do . v), dq = e k, dk = e q summed over the heads that share them, dg = 0.
    Sums of 16 terms and 64 heads, each rounding below 2^-24 of the terms: within 2^-17 of their sum."""
    import torch
    import selective_state_space_79_amd as ssm

    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    print("\n[gpu-case] delta gradients of 40000 sequences of one token", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(2)
    n, H, d, tol = 40000, 64, 16, 2.0 ** -17
    q, k = (torch.nn.functional.normalize(torch.randn(n, 1, d, generator=gen, device="cuda"), dim=-1) for _ in range(2))
    v, do = (torch.randn(n, H, d, generator=gen, device="cuda") for _ in range(2))
    g, beta = torch.zeros(n, H, device="cuda"), 0.1 + 0.9 * torch.rand(n, H, generator=gen, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    r = ssm.delta_bwd(q, k, v, g, beta, do=do, scale=0.5, cu_seqlens=cu)
    torch.cuda.synchronize()
    Q, K, V, O, B = (t.double() for t in (q, k, v, do, beta[..., None]))
    c, e, size = 0.5 * (Q * K).sum(-1, keepdim=True), 0.5 * (O * V * B).sum(-1, keepdim=True), 0.5 * (O * V * B).abs().sum(-1, keepdim=True)
    assert ((r["dv"].double() - B * c * O).abs() <= tol * (0.5 * B * O.abs())).all()
    assert ((r["dbeta"].double() - (c * (O * V).sum(-1, keepdim=True))[..., 0]).abs() <= tol * 0.5 * (O * V).abs().sum(-1)).all()
    for name, x in (("dq", K), ("dk", Q)):
        assert ((r[name].double() - e.sum(1, keepdim=True) * x).abs() <= tol * size.sum(1, keepdim=True)).all(), name
    assert (r["dg"].double().abs() <= tol * size[..., 0]).all()
