"""GPU: calls of the block operators that are allowed and rarer: rows as columns of a wider buffer
in every argument, batches with more than one leading dimension, heads that go two to a workgroup
over many chunks, the norms past 2^31 elements, on two streams at once and on expanded inputs."""
import sys

import pytest

from test_linattn_bounds_gpu import near
from test_linattn_gpu import Case, check_fwd, check_grads

pytestmark = pytest.mark.gpu


def announce(msg):
    print(f"\n[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("piece", [0, 128])
@pytest.mark.parametrize("dk,kheads,io", [(128, 1, "bf16"), (128, 24, "bf16"), (64, 1, "bf16"), (72, 2, "bf16"), (127, 1, "bf16"),
                                          (256, 1, "bf16"), (128, 1, "f32")])
def test_two_heads_to_a_workgroup_over_many_chunks(dk, kheads, io, piece):
    """More heads and pieces than CUs, one to four chunks, ends inside a chunk."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"two heads {dk} {kheads} {io} piece {piece}")
    c = Case([200, 129, 64, 1, 0, 70], 48, kheads, dk, 64, io, seed=dk + kheads)
    o, s = ssm.linattn_fwd(c.q, c.k, c.v, c.g, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, return_state=True, piece_len=piece)
    r = ssm.linattn_bwd(c.q, c.k, c.v, c.g, do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
    torch.cuda.synchronize()
    check_fwd(c, o, s)
    (ro, _), (ao, _) = c.ref_fwd(), c.ref_fwd(True)
    near("o", o, ro, ao, io, 2.0 ** -15)
    check_grads(c, r)


@pytest.mark.parametrize("pad", [0, 3, 8])
def test_batches_of_columns(pad):
    """(batch, L, heads, d) views of one projection: bitwise the packed tensors' results."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"batches of columns, pad {pad}")
    gen = torch.Generator(device="cuda").manual_seed(pad)
    B, L, H, d = 3, 90, 4, 64
    buf = torch.randn(B, L, 4 * H * d + pad, generator=gen, device="cuda").bfloat16()
    cut = lambda i: buf[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d))   # noqa: E731
    q, k, v, do = (cut(i) for i in range(4))
    g = -torch.rand(B, L, H, generator=gen, device="cuda")
    s0 = torch.randn(B, H, d, d, generator=gen, device="cuda")
    packed = [t.contiguous() for t in (q, k, v)]
    for piece in (0, 64):
        a, sa = ssm.linattn_fwd(q, k, v, g, s0=s0, return_state=True, piece_len=piece)
        b, sb = ssm.linattn_fwd(*packed, g, s0=s0, return_state=True, piece_len=piece)
        assert torch.equal(a, b) and torch.equal(sa, sb)
        x = ssm.linattn_bwd(q, k, v, g, do=do, s0=s0, piece_len=piece)
        y = ssm.linattn_bwd(*packed, g, do=do.contiguous(), s0=s0, piece_len=piece)
        assert all(torch.equal(x[n], y[n]) for n in y)
    # single tokens out of the same buffer
    pool, pool2 = s0.clone(), s0.clone()
    a = ssm.linattn_step(q[:, 5], k[:, 5], v[:, 5], g[:, 5].contiguous(), pool)
    b = ssm.linattn_step(*(t[:, 5].contiguous() for t in packed), g[:, 5].contiguous(), pool2)
    assert torch.equal(a, b) and torch.equal(pool, pool2)


@pytest.mark.parametrize("pad", [0, 3, 8])
def test_norms_of_columns_and_batches(pad):
    """(batch, L, dim) views, and strided x and r in the gradients: bitwise the packed results."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"norms of columns, pad {pad}")
    gen = torch.Generator(device="cuda").manual_seed(pad)
    B, L, D = 3, 50, 320
    buf = torch.randn(B, L, 4 * D + pad, generator=gen, device="cuda").bfloat16()
    x, z, res, dy = (buf[..., i * D:(i + 1) * D] for i in range(4))
    w, sc, po = (torch.randn(D, generator=gen, device="cuda") for _ in range(3))
    dyc = dy.contiguous()
    px, pz, pres = x.contiguous(), z.contiguous(), res.contiguous()
    y, r = ssm.add_norm_fwd(x, res, w, scale=sc, post_weight=po)
    y2, r2 = ssm.add_norm_fwd(px, pres, w, scale=sc, post_weight=po)
    assert torch.equal(y, y2) and torch.equal(r, r2) and y.shape == (B, L, D)
    wide = torch.zeros(B, L, D + 8 + pad, device="cuda", dtype=torch.bfloat16)
    rs = wide[..., :D]
    rs.copy_(r)
    a = ssm.add_norm_bwd(x, rs, w, dy=dyc, dr=dyc, scale=sc, post_weight=po)
    b = ssm.add_norm_bwd(px, r2, w, dy=dyc, dr=dyc, scale=sc, post_weight=po)
    assert all(torch.equal(a[n], b[n]) for n in b)
    for group, weight in ((D, w), (64, w), (64, w[:64].contiguous())):
        a = ssm.gated_norm_fwd(x, z, weight, group_size=group)
        assert torch.equal(a, ssm.gated_norm_fwd(px, pz, weight, group_size=group))
        a = ssm.gated_norm_bwd(x, z, weight, dy=dyc, group_size=group)
        b = ssm.gated_norm_bwd(px, pz, weight, dy=dyc, group_size=group)
        assert all(torch.equal(a[n], b[n]) for n in b)
    with pytest.raises(ValueError, match="contiguous"):
        ssm.add_norm_bwd(px, r2, w, dy=torch.ones((), device="cuda", dtype=torch.bfloat16).expand(B, L, D))


def test_norms_past_32_bits():
    """Rows past 2^31 elements: each row's results are those of a call of a few rows."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("norms past 32 bits")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    D, rows = 2048, (1 << 20) + 5
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, z, dy = (torch.randn(rows, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    assert x.numel() > 1 << 31
    w = torch.randn(D, generator=gen, device="cuda")
    few = slice(rows - 4, rows)
    y, r = ssm.add_norm_fwd(x, z, w, scale=w, post_weight=w)
    y2, r2 = ssm.add_norm_fwd(x[few], z[few], w, scale=w, post_weight=w)
    assert torch.equal(y[few], y2) and torch.equal(r[few], r2)
    a = ssm.add_norm_bwd(x, r, w, dy=dy, dr=z, scale=w, post_weight=w)
    b = ssm.add_norm_bwd(x[few], r2, w, dy=dy[few], dr=z[few], scale=w, post_weight=w)
    assert torch.equal(a["dx"][few], b["dx"]) and torch.equal(a["dresidual"][few], b["dresidual"])
    del a, y, r
    y = ssm.gated_norm_fwd(x, z, w, group_size=128)
    assert torch.equal(y[few], ssm.gated_norm_fwd(x[few], z[few], w, group_size=128))
    a = ssm.gated_norm_bwd(x, z, w, dy=dy, group_size=128)
    b = ssm.gated_norm_bwd(x[few], z[few], w, dy=dy[few], group_size=128)
    assert torch.equal(a["dx"][few], b["dx"]) and torch.equal(a["dz"][few], b["dz"])


def test_norms_on_two_streams_at_once():
    import torch
    import selective_state_space_79_amd as ssm

    announce("norms on two streams")
    gen = torch.Generator(device="cuda").manual_seed(4)
    sets = []
    for D in (1536, 4096):
        x, z, dy = (torch.randn(3000, D, generator=gen, device="cuda").bfloat16() for _ in range(3))
        sets.append((x, z, dy, torch.randn(D, generator=gen, device="cuda")))

    def calls(x, z, dy, w, stream=None):
        y, r = ssm.add_norm_fwd(x, z, w, post_weight=w, stream=stream)
        out = [y, r, *ssm.add_norm_bwd(x, z, w, dy=dy, post_weight=w, stream=stream).values()]
        return out + [ssm.gated_norm_fwd(x, z, w, stream=stream), *ssm.gated_norm_bwd(x, z, w, dy=dy, stream=stream).values()]

    want = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(sets):
            got[i].append(calls(*s, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))
