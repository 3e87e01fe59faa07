"""Gradients of the gated delta rule where a token keeps little or nothing of the state: the gradient of
a log decay g is then of the size of e^g, far below what the outputs' gradients are made of.

Bounds and their reasons are those of test_delta_gpu.py, of the norm of each head's dg: every term of dg
has the decays between as a factor, so that roundings are relative to them; a decay e^g is itself off
by 2^-24 |g| 1.44 at most, 2^-18 at g = -40.
"""
import numpy as np
import pytest

from test_delta_gpu import Case, announce, check_grads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,kheads,dk,dv,decay,piece", [
    ([150, 40], 2, 2, 64, 64, "token", 0),
    ([150, 40, 1, 0, 65], 4, 2, 128, 96, "token", 0),
    ([200], 2, 1, 256, 40, "token", 64),
    ([100, 33], 3, 1, 33, 77, "head", 0),
    ([64, 130], 2, 1, 128, 128, "head", 64),
    ([70] + [2, 1] * 300, 4, 2, 40, 64, "token", 0),      # heads on one q and k in turn
])
def test_gradients_of_fast_decays(lens, heads, kheads, dk, dv, decay, piece, io):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta fast decays {lens[:5]} {heads} {kheads} {dk} {dv} {decay} {piece} {io}")
    c = Case(lens, heads, kheads, dk, dv, io, decay, seed=dk)
    shape, rng = tuple(c.g.shape), np.random.default_rng(dk)
    for low, high in ((-3, -3), (-6, -6), (-10, -10), (-20, -20), (-40, -40), (-12, -6)):
        c.g = torch.from_numpy(rng.uniform(low, high, shape).astype(np.float32)).cuda()
        r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
        torch.cuda.synchronize()
        print("decays", low, high, flush=True)
        check_grads(c, r)
    # nothing at all is kept: nothing depends on the decay
    c.g = torch.full(shape, float("-inf"), device="cuda")
    r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
    torch.cuda.synchronize()
    assert (r["dg"].abs() < 1e-37).all() and (r["ds0"][[i for i, n in enumerate(lens) if n]].abs() < 1e-37).all()
    check_grads(c, r)
