"""GPU: every operand of linear attention's products is held to float32, whatever the call
asks for and whatever type its rows have.

Terms that all but cancel show what each operand lost: the outputs are small, so their own
rounding is, and what remains is a share of the terms.

Bounds of the cancelling terms, as shares of A, the sum of the terms' absolute values.  An
output has at most 2 terms per product, 3 parts of an operand each (6 additions), and an
addition inside the matrix unit is off by at most 2^-23 of the running sum (it may truncate):
6 * 2^-23.  A decay is one exponential (2^-23) of a difference of sums that two floats hold,
times the scale, times the product (2^-24 each), and three bf16 parts leave out at most 2^-25
of a value: together below 2^-21.  In all less than 2^-19 A, where two bf16 parts alone may
leave out 2^-18 A.  A bf16 output is rounded by at most 2^-8 of its value.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SHARE = 2.0 ** -19


def announce(msg):
    print(f"\n[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


def dtype(io):
    import torch

    return torch.bfloat16 if io == "bf16" else torch.float32


# heads and columns of the kernels' shapes: whole heads, two narrow heads that share q and k
# (more of them than the card has CUs), narrow heads of their own; 64, 128 and 256 state rows
SHAPES = [(64, 64, 2, 128), (300, 1, 2, 64), (64, 64, 2, 64), (300, 1, 66, 64), (64, 64, 66, 128), (300, 1, 130, 64),
          (64, 64, 130, 128)]


def inputs(io, heads, kheads, T, dk, dv, seed):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    q, k = torch.zeros(T, kheads, dk, device="cuda"), torch.zeros(T, kheads, dk, device="cuda")
    v = torch.zeros(T, heads, dv, device="cuda")
    g = torch.zeros(T, heads, device="cuda")
    return rnd, q, k, v, g


def run(ssm, io, q, k, v, g, **kw):
    t = dtype(io)
    return ssm.linattn_fwd(q.to(t), k.to(t), v.to(t), g, **kw)


def held(got, want, terms, io):
    over = (got.double() - want).abs() / (HALF[io] * want.abs() + SHARE * terms + 1e-30)
    assert bool(got.isfinite().all())
    assert float(over.max()) <= 1, f"{float(over.max()):.3g} of the bound"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kheads,dk,dv", SHAPES)
def test_state_at_the_read_out(heads, kheads, dk, dv, io):
    """o = q . S of two state rows that differ by 2^-13 of themselves."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"state {heads} {kheads} {dk} {dv} {io}")
    rnd, q, k, v, g = inputs(io, heads, kheads, 1, dk, dv, 1)
    a = rnd(1, heads, dv)
    s0 = torch.zeros(1, heads, dk, dv, device="cuda")
    s0[:, :, 0], s0[:, :, -1] = a, a * (1 + 2.0 ** -13 * rnd(1, heads, dv))
    q[:, :, 0], q[:, :, -1] = 1.0, -1.0
    o = run(ssm, io, q, k, v, g, s0=s0)
    x, y = s0[:, :, 0].double(), s0[:, :, -1].double()
    held(o, x - y, x.abs() + y.abs(), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kheads,dk,dv", SHAPES)
def test_products_inside_a_chunk(heads, kheads, dk, dv, io):
    """o_1 = (q . k) (e^g v_0 + v_1) with v_1 = -v_0 and a decay of about 2^-11: the product of
    a bf16 query and key has 16 bits, its decayed value all 24.  In every tile of a chunk of 64
    tokens: the pair lies at tokens i and j."""
    import torch
    import selective_state_space_79_amd as ssm

    T = 64
    for i, j in ((0, 1), (3, 20), (15, 40), (2, 63), (17, 18), (20, 47), (18, 60), (33, 40), (40, 60), (50, 63)):
        if io == "f32" and (i < 32) != (j < 32):
            continue    # chunks of 32 tokens: the pair meets in the state
        announce(f"chunk {heads} {kheads} {dk} {dv} {io} {i} {j}")
        rnd, q, k, v, g = inputs(io, heads, kheads, T, dk, dv, 2)
        q[j, :, 0], k[i, :, 0] = rnd(kheads).bfloat16().float(), rnd(kheads).bfloat16().float()
        k[j] = k[i]
        v[i] = rnd(heads, dv).bfloat16().float()
        v[j] = -v[i]
        g[j] = -(2.0 ** -11) * (0.5 + rnd(heads).abs())
        o = run(ssm, io, q, k, v, g)
        qk = (q[j, :, 0].double() * k[i, :, 0].double()).repeat_interleave(heads // kheads)[:, None]
        x, y = qk * torch.exp(g[j].double())[:, None] * v[i].double(), qk * v[j].double()
        held(o[j], x + y, x.abs() + y.abs(), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("piece", [0, 64])
@pytest.mark.parametrize("heads,kheads,dk,dv", SHAPES)
def test_rows_that_the_state_takes(heads, kheads, dk, dv, piece, io):
    """S = k (f v_0 + v_1) with v_1 = -v_0 and f about 1 - 2^-11, read by a token of the next
    chunk (or piece): the decayed value row has all 24 bits.  No final state is asked for."""
    import torch
    import selective_state_space_79_amd as ssm

    T = 70
    announce(f"state rows {heads} {kheads} {dk} {dv} {io} piece {piece}")
    rnd, q, k, v, g = inputs(io, heads, kheads, T, dk, dv, 3)
    q[68, :, 0], k[5, :, 0] = 1.0, rnd(kheads).bfloat16().float()
    k[9] = k[5]
    v[5] = rnd(heads, dv).bfloat16().float()
    v[9] = -v[5]
    g[9] = -(2.0 ** -11) * (0.5 + rnd(heads).abs())
    g[20] = -0.25
    o = run(ssm, io, q, k, v, g, piece_len=piece)
    kk = k[5, :, 0].double().repeat_interleave(heads // kheads)[:, None] * torch.exp(g[20].double())[:, None]
    x, y = kk * torch.exp(g[9].double())[:, None] * v[5].double(), kk * v[9].double()
    # the state's scale and its split at the read-out are one step of each kind more
    held(o[68], x + y, 1.5 * (x.abs() + y.abs()), io)


@pytest.mark.parametrize("piece", [0, 64])
@pytest.mark.parametrize("heads,kheads,dk,dv", SHAPES)
def test_outputs_do_not_depend_on_the_states_asked_for(heads, kheads, dk, dv, piece):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"with and without states {heads} {kheads} {dk} {dv} piece {piece}")
    gen = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()   # noqa: E731
    q, k, v = rnd(200, kheads, dk), rnd(200, kheads, dk), rnd(200, heads, dv)
    g = -torch.rand(200, heads, generator=gen, device="cuda")
    a = ssm.linattn_fwd(q, k, v, g, piece_len=piece)
    b, _ = ssm.linattn_fwd(q, k, v, g, piece_len=piece, return_state=True)
    assert torch.equal(a, b)
