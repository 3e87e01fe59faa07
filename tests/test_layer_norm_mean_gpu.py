"""Layer norm where the mean is large beside the deviations: rows of equal values have no
deviation, whatever the value, and a mean far from zero leaves the deviations their digits.

Bounds.  A mean held as two floats leaves no term of size |x| but its second rounding, 2^-48 of it.
A sum over a row passes at most 26 additions (8 or 16 values a thread, 6 steps over a wave's lanes, 4
over 16 waves), each rounded by 2^-24 of the terms' absolute sum.  A deviation d is off by two
roundings of its own, and by what a mean summed in float32 within a thread may lack where the values are
of unlike size, so that the deviations are as large as they: 2^-24 of 28 (mean |d| + |d|) in all; the
reciprocal of its root mean square by 20 roundings, a value of y = d rs w by less than 2^-18 of (|d| +
mean |d|) rs |w|.  dx = rs (u - mean u - n mean (u n)) with u = dy w and n = d rs takes n twice, rs
three times and three such sums: 2^-17 of its terms' absolute values, with |n| + mean |n| for n.  Weight
gradients add up to 64 rows here, each addition rounded by 2^-24 of the absolute sum: 2^-18 of that once
more.
"""
import numpy as np
import pytest

import delta_ref as ref
from test_layer_norm_gpu import EPS, HALF, announce, dtype, host, put

pytestmark = pytest.mark.gpu


def bounds(x, w, dy, io):
    """Largest allowed errors of y, dx and dweight, and the float64 values themselves."""
    d = x - x.mean(-1, keepdims=True)
    rs = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + EPS)
    mean = lambda t: np.abs(t).mean(-1, keepdims=True)   # noqa: E731
    rest = 2.0 ** -24 * np.abs(x).max(-1, keepdims=True)
    n, u = d * rs, dy * w
    wide = np.abs(n) + mean(n) + rest * rs
    want = dict(y=ref.layer_norm(x, w, None, EPS), **ref.layer_norm_grads(x, w, dy, EPS))
    room = dict(y=2.0 ** -18 * wide * np.abs(w),
                dx=2.0 ** -17 * rs * (np.abs(u) + mean(u) + wide * (mean(u * n) + mean(u) * mean(n))),
                dweight=2.0 ** -18 * (np.abs(dy) * (wide + np.abs(n))).sum(0))
    for name in ("y", "dx"):
        room[name] = room[name] + HALF[io] * np.abs(want[name])
    # what the checks have to notice: a gradient without one of its parts, or none at all
    drop = dict(nothing=np.zeros_like(u), mean=rs * (u - n * (u * n).mean(-1, keepdims=True)), n=rs * (u - u.mean(-1, keepdims=True)))
    for part, other in drop.items():
        over = np.abs(other - want["dx"]) / room["dx"]
        assert np.median(over.max(-1)) > 4, (part, np.median(over.max(-1)))
    return want, room


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim,far", [(50, 768, 1000.0), (7, 1535, -3000.0), (40, 64, 500.0), (64, 72, 1e5), (5, 4096, 1000.0),
                                          (4, 8200, 200.0), (3, 16384, -1000.0), (60, 7, 100.0)])
def test_a_mean_far_from_zero_costs_no_digits(rows, dim, far, io):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"layer norm {rows} x {dim} around {far} {io}")
    rng = np.random.default_rng(dim)
    # in bf16 values around `far` are 2^-8 of it apart at the nearest: deviations of that size
    x = put(rng, rows, dim, io=io, mul=1.0 if io == "f32" else abs(far) * 2.0 ** -5, add=far)
    dy, w = put(rng, rows, dim, io=io, add=0.5), put(rng, dim, mul=0.2, add=1.0)
    want, room = bounds(host(x), host(w), host(dy), io)
    y = ssm.layer_norm_fwd(x, w, eps=EPS)
    r = ssm.layer_norm_bwd(x, w, dy=dy, eps=EPS)
    torch.cuda.synchronize()
    for name, got in (("y", y), ("dx", r["dx"]), ("dweight", r["dweight"])):
        over = np.abs(host(got) - want[name]) / room[name]
        assert over.max() <= 1, f"{name}: {over.max():.3g} of the bound"


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_of_equal_values_are_the_bias(io):
    """A mean rounded to float32 from a sum in float32 is off by a few units of its last place, and so
    were all deviations: y 0.7 off for three values of 1.7e9, 0.014 for three of 1000.1."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"layer norm equal values {io}")
    for dim in (1, 3, 100, 768, 1535, 2048, 4095, 8192, 16383):
        x = torch.tensor([0.1, 1000.1, -1e5 / 7, 3e-3, 1.7e9, -5e-20, 0.3], device="cuda").to(dtype(io))[:, None].expand(7, dim).contiguous()
        w, b = torch.full((dim,), 0.7, device="cuda"), torch.full((dim,), 0.25, device="cuda")
        for eps in (1e-5, 2.0 ** -126):
            y = ssm.layer_norm_fwd(x, w, b, eps=eps)
            r = ssm.layer_norm_bwd(x, w, dy=torch.ones_like(x), eps=eps)
            torch.cuda.synchronize()
            assert (y == 0.25).all(), (dim, eps, (y.float() - 0.25).abs().amax(1))
            assert torch.isfinite(r["dx"]).all() and (r["dbias"] == 7).all() and (r["dweight"] == 0).all(), (dim, eps)
