"""The gated delta rule over sequences long enough that the library cuts them itself, and over packs of
one long and many short sequences, against the float64 recurrence in both types.

Bounds and their reasons are those of test_delta_gpu.py.  Decays are slow in some heads, so that what
crosses the pieces' joints counts; with steps of 0.1 to 0.9 a state of at most 128 keys forgets a
direction by half in 180 tokens at the mean step, and errors older than 512 tokens have gone: 2e5
roundings of random sign, 452 * 2^-25 < 2^-16 of the norm, whatever the length.
"""
import numpy as np
import pytest

from test_delta_gpu import Case, announce, check_fwd, check_grads
from test_delta_pieces_gpu import slow

pytestmark = pytest.mark.gpu


def workspace(c, back, piece):
    import selective_state_space_79_amd as ssm

    d = ssm.blocks._delta_dims(*c.rows(), c.scale, c.n)
    d.piece_len = piece
    return (ssm.ssm_delta_bwd_workspace_bytes if back else ssm.ssm_delta_fwd_workspace_bytes)(d)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,kheads,dk,dv,decay,pieces", [
    ([2100], 2, 1, 128, 96, "token", (0,)),
    ([1500, 900], 4, 2, 100, 64, "head", (0,)),
    ([1900], 3, 3, 72, 40, "token", (0,)),
    # too short on average for the library to cut them by itself
    ([1700, 5, 0, 64, 1, 33, 65, 2, 128, 1, 7, 31], 2, 1, 128, 96, "token", (0, 256)),
    ([3, 64, 16, 1300, 1, 0, 90, 40], 3, 1, 64, 128, "head", (0, 192)),
])
def test_long_sequences(lens, heads, kheads, dk, dv, decay, pieces, io):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta long {lens} {heads} {kheads} {dk} {dv} {decay} {io}")
    c = slow(Case(lens, heads, kheads, dk, dv, io, decay, seed=sum(lens)), np.random.default_rng(len(lens)))
    for back in (False, True):
        cut = [workspace(c, back, piece) > workspace(c, back, 1 << 20) for piece in pieces]
        assert cut == ([True] if len(pieces) == 1 else [False, True])
    want_fwd, want_bwd = c.ref_fwd(), c.ref_bwd()
    c.ref_fwd, c.ref_bwd = lambda: want_fwd, lambda: want_bwd
    for piece in pieces:
        kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0, piece_len=piece)
        o, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
        r = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw)
        torch.cuda.synchronize()
        check_fwd(c, o, s)
        check_grads(c, r)
