"""GPU: linear attention at the ends of the sizes that its entry points allow."""
import sys

import pytest

pytestmark = pytest.mark.gpu


def announce(msg):
    print(f"\n[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("heads,dk,io", [(20000, 248, "bf16"), (32767, 130, "bf16"), (32767, 255, "f32")])
def test_gradients_of_very_many_heads(heads, dk, io):
    """Rows of all heads up to 33 MB: every head's gradients are bitwise those of a call with a
    few heads (which test_linattn_gpu.py compares with float64)."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"many heads {heads} {dk} {io}")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    T, dv = 64, 16 if io == "bf16" else 8
    t = torch.bfloat16 if io == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(heads)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(t)   # noqa: E731
    q, k, v, do = rnd(T, heads, dk), rnd(T, heads, dk), rnd(T, heads, dv), rnd(T, heads, dv)
    g = -torch.rand(T, heads, generator=gen, device="cuda")
    r = ssm.linattn_bwd(q, k, v, g, do=do)
    torch.cuda.synchronize()
    for h in (0, 1, heads // 3, heads // 2 + 1, heads - 40):
        announce(f"heads from {h}")
        part = [x[:, h:h + 40].contiguous() for x in (q, k, v, g, do)]
        want = ssm.linattn_bwd(*part[:4], do=part[4])
        for name in want:
            assert torch.equal(r[name][:, h:h + 40], want[name]), name
