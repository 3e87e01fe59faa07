"""GPU parity of the norms around a block (ssm_gated_norm_*, ssm_add_norm_*) against the
float64 rows of block_ref.py.

Bounds.  Every value passes a handful of float32 roundings and the hardware's reciprocal
square root, exponential and reciprocal (one unit each): 16 roundings of 2^-24 and a sum of
n squares in a tree, together below 2^-18 of the value's own terms.  A gradient at a row is a
difference, so its bound is taken of both of its parts; sums over rows add 2^-24 for each
row in the worst order, and are taken of the terms' absolute sum.  A bf16 output is rounded
by at most 2^-8 of its value.
"""
import sys

import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TERM = 2.0 ** -18
EPS = 1e-5


def announce(msg):
    print(f"\n[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


def dtype(io):
    import torch

    return torch.bfloat16 if io == "bf16" else torch.float32


def put(rng, *shape, io="f32", mul=1.0, add=0.0):
    import torch

    return torch.from_numpy((rng.standard_normal(shape) * mul + add).astype(np.float32)).cuda().to(dtype(io))


def host(t):
    return None if t is None else t.double().cpu().numpy()


def check(name, got, want, terms, io):
    got = host(got)
    assert np.isfinite(got).all(), name
    over = np.abs(got - want) / (HALF[io] * np.abs(want) + TERM * np.maximum(terms, np.abs(want)) + 1e-30)
    assert over.max() <= 1, f"{name}: {over.max():.3g} of the bound at {np.unravel_index(over.argmax(), over.shape)}"


def parts(dn, x, eps):
    """Absolute size of the two parts of a norm's gradient."""
    r = ref.rms(x, eps)
    n = np.abs(x * r)
    return r * (np.abs(dn) + n * (np.abs(dn) * n).mean(-1, keepdims=True))


GATED = [(1, 1, 1), (3, 1, 7), (5, 3, 64), (33, 4, 128), (9, 2, 200), (7, 1, 1536), (300, 64, 64), (4, 1, 4096), (3, 1, 8200),
         (2, 1, 16384), (1200, 1, 72), (5, 2, 2048), (2100, 1, 640)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("rows,groups,group", GATED)
def test_gated_norm(rows, groups, group, first, io):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"gated norm {rows} {groups}x{group} first={first} {io}")
    rng = np.random.default_rng(rows + group)
    dim = groups * group
    for shared in ([False, True] if groups > 1 else [False]):
        for gate in (True, False):
            x, dy = put(rng, rows, dim, io=io, mul=2.0), put(rng, rows, dim, io=io)
            z = put(rng, rows, dim, io=io) if gate else None
            w = put(rng, group if shared else dim, mul=0.2, add=1.0)
            kw = dict(group_size=group, gate_first=first, eps=EPS)
            y = ssm.gated_norm_fwd(x, z, w, **kw)
            r = ssm.gated_norm_bwd(x, z, w, dy=dy, **kw)
            torch.cuda.synchronize()
            hx, hz, hw, hd = host(x), host(z), host(w), host(dy)
            want = ref.gated_norm(hx, hz, hw, group, first, EPS)
            check("y", y, want, np.abs(want), io)
            g = ref.gated_norm_grads(hx, hz, hw, hd, group, first, EPS)
            shape = (rows, groups, group)
            a = np.ones(shape) if hz is None else ref.silu(hz.reshape(shape))
            zz = np.zeros(shape) if hz is None else hz.reshape(shape)
            sg = 1 / (1 + np.exp(-zz))
            slope = np.abs(sg) * (1 + np.abs(zz) * (1 - sg))
            xs, ds = hx.reshape(shape), hd.reshape(shape)
            p = xs * a if first else xs
            up = ds if first else ds * a
            wf = np.broadcast_to(hw.reshape(-1, group), shape[1:])
            dp = parts(up * wf, p, EPS)
            n = np.abs(p * ref.rms(p, EPS))
            check("dx", r["dx"], g["dx"], (dp * np.abs(a) if first else dp).reshape(rows, dim), io)
            if gate:
                check("dz", r["dz"], g["dz"], ((dp * np.abs(xs) if first else np.abs(ds) * n * np.abs(wf)) * slope)
                      .reshape(rows, dim), io)
            dw = (np.abs(up) * n).sum(0)
            check("dweight", r["dweight"], g["dweight"], (dw.sum(0) if shared else dw).reshape(-1), "f32")


ADD = [(1, 1), (3, 7), (5, 64), (2, 130), (33, 1536), (4, 4096), (9, 2048), (3, 8200), (2, 16384), (1100, 96), (2050, 520)]


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("post,scale", [(False, False), (True, False), (False, True), (True, True)])
def test_add_norm(post, scale, io, res):
    import torch
    import selective_state_space_79_amd as ssm

    for rows, dim in ADD:
        announce(f"add norm {rows}x{dim} post={post} scale={scale} {io}/{res}")
        rng = np.random.default_rng(rows + dim)
        x, dy = put(rng, rows, dim, io=io), put(rng, rows, dim, io=io)
        s, dr = put(rng, rows, dim, io=res, mul=2.0), put(rng, rows, dim, io=res)
        w = put(rng, dim, mul=0.2, add=1.0)
        sc = put(rng, dim, mul=0.3, add=0.5) if scale else None
        po = put(rng, dim, mul=0.2, add=1.0) if post else None
        y, r = ssm.add_norm_fwd(x, s, w, scale=sc, post_weight=po, eps=EPS)
        gr = ssm.add_norm_bwd(x, r, w, dy=dy, dr=dr, scale=sc, post_weight=po, eps=EPS)
        torch.cuda.synchronize()
        hx, hs, hw, hsc, hpo, hdy, hdr, hr = map(host, (x, s, w, sc, po, dy, dr, r))
        # y is the norm of r as stored: take the stored r itself
        wy, wr, _ = ref.add_norm(hx, hs, hw, hsc, hpo, EPS, lambda v: hr)
        a = hx * ref.rms(hx, EPS) * hpo if post else hx
        check("r", r, wr, np.abs(hs) + np.abs(a if hsc is None else a * hsc), res)
        check("y", y, wy, np.abs(wy), io)
        want = ref.add_norm_grads(hx, hr, hw, hdy, hdr, hsc, hpo, EPS)
        d = parts(hdy * hw, hr, EPS) + np.abs(hdr)
        check("dresidual", gr["dresidual"], want["dresidual"], d, res)
        check("dweight", gr["dweight"], want["dweight"], np.abs(hdy * hr * ref.rms(hr, EPS)).sum(0), "f32")
        n = np.abs(hx * ref.rms(hx, EPS)) if post else np.abs(hx)
        if scale:
            check("dscale", gr["dscale"], want["dscale"], (d * (n * np.abs(hpo) if post else n)).sum(0), "f32")
            d = d * np.abs(hsc)
        if post:
            check("dpost_weight", gr["dpost_weight"], want["dpost_weight"], (d * n).sum(0), "f32")
            d = parts(d * np.abs(hpo), hx, EPS)
        check("dx", gr["dx"], want["dx"], d, io)


def test_add_norm_without_residual_or_gradient_from_behind():
    import torch
    import selective_state_space_79_amd as ssm

    announce("add norm, no residual")
    rng = np.random.default_rng(3)
    x, dy, w = put(rng, 6, 320, io="bf16"), put(rng, 6, 320, io="bf16"), put(rng, 320, add=1.0)
    y, r = ssm.add_norm_fwd(x, None, w, eps=EPS)
    assert torch.equal(r, x)
    a = ssm.add_norm_bwd(x, r, w, dy=dy, eps=EPS)
    b = ssm.add_norm_bwd(x, r, w, dy=dy, dr=torch.zeros_like(r), eps=EPS)
    for name in a:
        assert torch.equal(a[name], b[name]), name
    f = torch.empty(6, 320, device="cuda")
    ssm.add_norm_fwd(x, None, w, eps=EPS, residual_out=f)
    assert torch.equal(f, x.float())


def test_in_place_and_strided_rows():
    """r over the residual, y over x or z, rows as columns of a wider buffer (also with steps
    that allow no 16-byte access): bitwise what packed rows give."""
    import torch
    import selective_state_space_79_amd as ssm

    rng = np.random.default_rng(5)
    for pad in (0, 8, 3):
        announce(f"strided norms, pad {pad}")
        x, z, s = (put(rng, 50, 256, io="bf16") for _ in range(3))
        w = put(rng, 256, add=1.0)
        y, r = ssm.add_norm_fwd(x, s, w, eps=EPS)
        buf = torch.zeros(50, 3 * 256 + pad, dtype=torch.bfloat16, device="cuda")
        xs, ss, ys = buf[:, :256], buf[:, 256:512], buf[:, 512 + pad:]
        xs.copy_(x), ss.copy_(s)
        y2, r2 = ssm.add_norm_fwd(xs, ss, w, eps=EPS, residual_out=ss, out=ys)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(r, r2) and torch.equal(buf[:, 256:512], r)
        g = ssm.gated_norm_fwd(x, z, w, eps=EPS)
        gb = ssm.gated_norm_bwd(x, z, w, dy=x, eps=EPS)
        ss.copy_(z)
        g2 = ssm.gated_norm_fwd(xs, ss, w, eps=EPS, out=ss).clone()
        ss.copy_(z)
        gb2 = ssm.gated_norm_bwd(xs, ss, w, dy=x, eps=EPS)
        torch.cuda.synchronize()
        assert torch.equal(g, g2)
        assert all(torch.equal(gb[n], gb2[n]) for n in gb)


def test_norms_captured_and_replayed():
    import torch
    import selective_state_space_79_amd as ssm

    announce("norms in a graph")
    rng = np.random.default_rng(6)
    x, s, dy = (put(rng, 700, 512, io="bf16") for _ in range(3))
    w = put(rng, 512, add=1.0)
    st = torch.cuda.Stream()

    def calls():
        y, r = ssm.add_norm_fwd(x, s, w, scale=w, post_weight=w)
        a = ssm.add_norm_bwd(x, r, w, dy=dy, scale=w, post_weight=w)
        b = ssm.gated_norm_bwd(x, s, w[:128], dy=dy, group_size=128)
        return [y, r, ssm.gated_norm_fwd(x, s, w)] + list(a.values()) + list(b.values())

    calls()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got = calls()
    for _ in range(4):
        x.add_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, calls()))


def test_extreme_rows():
    """Rows of zeros, rows with large and tiny values, gates far on both sides."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("extreme rows")
    x = torch.zeros(4, 64, device="cuda")
    x[1], x[2], x[3, 0] = 1e15, 1e-15, 1.0
    z = torch.full((4, 64), 80.0, device="cuda")
    z[:, 1::2] = -200.0
    w = torch.ones(64, device="cuda")
    for first in (True, False):
        y = ssm.gated_norm_fwd(x, z, w, gate_first=first, eps=EPS)
        r = ssm.gated_norm_bwd(x, z, w, dy=torch.ones_like(x), gate_first=first, eps=EPS)
        torch.cuda.synchronize()
        want = ref.gated_norm(host(x), host(z), host(w), 64, first, EPS)
        check("y", y, want, np.abs(want) + 1e-20, "f32")
        assert all(bool(t.isfinite().all()) for t in r.values())
    y, r = ssm.add_norm_fwd(x, x, w, eps=EPS)
    assert bool(y.isfinite().all())
