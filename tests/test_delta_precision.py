"""The gated delta rule's products are held to float32: operands that are no bf16 inputs go into them in
three bf16 parts.  The bounds here are between what that leaves and what two parts would.

Bounds.  A value passes, in each chunk of 32 tokens, up to 256 / 32 steps of the matrix unit over the
state's rows and three over the chunk's tokens, six products of parts each: 66 roundings, each of 2^-24
of the partial sum at most, 2^-25 in the mean square, of random sign.  Over 300 tokens and no more
decay than that, 10 chunks: 660, whose root times 2^-25 is 8e-7 < 2^-20 of the head's norm (FINE).  A
gradient passes the same twice: 2^-19.  Cut to two parts an operand lacks up to 2^-17 of itself, 2^-18
in the mean square, in five operands a chunk: a model of the walks in float64 with nothing but these
cuts leaves the bounds (on the CPU), and with three parts stays an eighth of the way to them.
"""
import numpy as np
import pytest

import delta_ref as ref
from test_delta_gpu import Case, announce
from test_delta_pieces_gpu import slow

FINE = 2.0 ** -20

CASES = [
    # lens, heads, dk, dv, io, slow decays
    ([300], 2, 128, 128, "f32", False),
    ([300], 2, 128, 128, "f32", True),
    ([130, 33, 64], 3, 64, 64, "f32", True),
    ([200, 90], 2, 256, 100, "f32", False),
    ([200, 90], 2, 96, 250, "f32", True),
    ([150], 4, 33, 77, "f32", False),
    ([300], 2, 128, 128, "bf16", True),
    ([300], 2, 64, 64, "bf16", False),
    ([300], 2, 160, 64, "bf16", False),
]
IDS = ["-".join(str(x).replace(" ", "") for x in c) for c in CASES]


def make(lens, heads, dk, dv, io, slowly):
    c = Case(lens, heads, heads, dk, dv, io, seed=len(str(lens)) + dk)
    return slow(c, np.random.default_rng(dk)) if slowly else c


def off(got, want):
    """The error's norm over the value's, the largest over the heads (axis 1)."""
    axes = tuple(i for i in range(want.ndim) if i != 1)
    return (np.sqrt(((got - want) ** 2).sum(axes)) / np.sqrt((want ** 2).sum(axes))).max()


def cut(x, parts):
    """x in bf16 parts, added up."""
    left, total = x.astype(np.float32), np.zeros(x.shape)
    for _ in range(parts):
        bits = left.view(np.uint32).astype(np.uint64)
        one = ((bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
        total, left = total + one, left - one
    return total


def model(c, parts):
    """Both walks in chunks of 32 tokens, in float64 but for the operands' parts: o, s_last, dv, ds0."""
    q, k, v, g, beta, scale, starts = c.args()
    do, s0, dsl, P = c.host(c.do), c.host(c.s0), c.host(c.ds_last), lambda x: cut(x, parts)
    if c.io == "f32":
        q, k, v, do = (P(x) for x in (q, k, v, do))
    out = dict(o=np.zeros_like(v), s_last=np.zeros_like(s0), dv=np.zeros_like(v), ds0=np.zeros_like(s0))
    for h in range(v.shape[1]):
        for n in range(len(starts) - 1):
            S, dS = s0[n, h], dsl[n, h]
            chunks = [slice(a, min(a + 32, starts[n + 1])) for a in range(starts[n], starts[n + 1], 32)]

            def parts_of(t):
                G = np.cumsum(g[t, h])
                L = np.tril(np.exp(np.minimum(G[:, None] - G[None, :], 0)))
                A = np.linalg.inv(np.eye(len(G)) + beta[t, h][:, None] * np.tril(L * (k[t, h] @ k[t, h].T), -1))
                return np.exp(G)[:, None], np.exp(G[-1] - G)[:, None], P(A), P(scale * L * (q[t, h] @ k[t, h].T)), beta[t, h][:, None]

            for t in chunks:
                e, tail, A, D, b = parts_of(t)
                U = A @ P(b * (v[t, h] - e * (k[t, h] @ P(S))))
                out["o"][t, h] = scale * e * (q[t, h] @ P(S)) + D @ P(U)
                S = e[-1] * S + k[t, h].T @ P(tail * U)
            for t in reversed(chunks):
                e, tail, A, D, b = parts_of(t)
                Z = A.T @ P(D.T @ do[t, h] + tail * (k[t, h] @ P(dS)))
                out["dv"][t, h] = b * Z
                dS = e[-1] * dS + q[t, h].T @ P(scale * e * do[t, h]) - k[t, h].T @ P(e * b * Z)
            out["s_last"][n, h], out["ds0"][n, h] = S, dS
    return out


def wanted(c):
    o, s = c.ref_fwd()
    return dict(o=o, s_last=s, **c.ref_bwd())


def on_cpu(monkeypatch):
    import torch

    monkeypatch.setattr(torch.Tensor, "cuda", lambda self, *a, **k: self)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_bounds_tell_two_parts_from_three(case, monkeypatch):
    on_cpu(monkeypatch)
    c = make(*case)
    want, two, three = wanted(c), model(c, 2), model(c, 3)
    for name, bound in (("o", FINE), ("s_last", FINE), ("dv", 2 * FINE), ("ds0", 2 * FINE)):
        a, b = off(two[name], want[name]), off(three[name], want[name])
        assert a > 1.25 * bound and b < bound / 8, f"{name}: two parts {a:.3g}, three {b:.3g} of {bound:.3g}"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_outputs_are_held_to_float32(case):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta precision {case}")
    c = make(*case)
    want, s_want = c.ref_fwd()
    for piece in (0, 64):
        o, s = ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s0=c.s0, return_state=True, piece_len=piece)
        torch.cuda.synchronize()
        got = [("s_last", off(c.host(s), s_want))] + ([("o", off(c.host(o), want))] if c.io == "f32" else [])
        print(piece, *got, flush=True)
        assert all(x <= FINE for _, x in got), got


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradients_are_held_to_float32(case):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta gradients' precision {case}")
    c = make(*case)
    want = c.ref_bwd()
    for piece in (0, 64):
        r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
        torch.cuda.synchronize()
        names = ("dq", "dk", "dv", "ds0", "dbeta") if c.io == "f32" else ("ds0", "dbeta")
        got = [(n, off(c.host(r[n]), want[n])) for n in names]
        print(piece, *got, flush=True)
        assert all(x <= 2 * FINE for _, x in got), got
