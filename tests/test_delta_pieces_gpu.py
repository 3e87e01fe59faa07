"""Pieces of the gated delta rule where what crosses a joint counts: slow decays and small steps, so
that a state lives through several pieces and a piece's transition (what it makes of the state that it
starts from) is neither zero nor the unit matrix.

Bounds and their reasons are those of test_delta_gpu.py: no step makes a state or an error in one
longer (keys of length 0.99 at most, 0 < beta < 1, decays of at most one).  A state here forgets by its
steps, a direction of dk by 1 - beta / dk a token, so that errors live for dk / beta <= 512 tokens and
2e5 roundings of random sign add up to 452 * 2^-25 < 2^-16 of the norm.  Each case also shows, from
the float64 recurrence alone, that results would leave their bounds if a joint took its piece's own end
state without the transition, at the first joint or at a later one.
"""
import numpy as np
import pytest

import delta_ref as ref
from test_delta_gpu import HALF, NORM, Case, announce, check_fwd, check_grads

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "ds0")


def slow(c, rng):
    """Decays of 0 to 1e-3 in the even heads, none in the odd ones; steps inside 0.1 .. 0.9."""
    import torch

    g = -1e-3 * rng.random(tuple(c.g.shape))
    g[..., 1::2] = 0.0
    c.g = torch.from_numpy(g.astype(np.float32)).to(c.g.device)
    c.beta = torch.from_numpy(rng.uniform(0.1, 0.9, tuple(c.beta.shape)).astype(np.float32)).to(c.beta.device)
    return c


def beyond(want, other, half, times=1):
    """How far `other` leaves check()'s bound of the norm, the largest over the heads (axis 1)."""
    rest = np.maximum(np.abs(other - want) - half * np.abs(want), 0)
    axes = tuple(i for i in range(want.ndim) if i != 1)
    return (np.sqrt((rest ** 2).sum(axes)) / (times * NORM * np.sqrt((want ** 2).sum(axes)) + 1e-30)).max()


def joints_count(c, piece, back):
    """Sequence 0 in pieces, each from the state (and, against time, the gradient) that the ones beside it
    leave: once joined as they are, and once with one joint that drops the transition."""
    q, k, v, g, beta, scale, starts = c.args()
    cut = list(range(int(starts[0]), int(starts[1]), piece)) + [int(starts[1])]
    n = len(cut) - 1
    assert n >= 4
    part = lambda i: ([q, k, v, g, beta, scale, np.array(cut[i:i + 2])], slice(cut[i], cut[i + 1]))   # noqa: E731
    zero = np.zeros_like(c.host(c.s0)[:1])
    end = lambda i, s: ref.delta(*part(i)[0], s)[1]      # noqa: E731
    do = c.host(c.do)
    start = lambda i, s, ds: ref.delta_grads(*part(i)[0], do, s, ds)      # noqa: E731

    def joined(drop=None, drop_back=None):
        s = [c.host(c.s0)[:1]]
        for i in range(n):
            s.append(end(i, zero if i == drop else s[i]))
        if not back:
            o = np.concatenate([ref.delta(*part(i)[0], s[i])[0][part(i)[1]] for i in range(n)])
            return dict(o=o, s_last=s[n])
        ds, out = c.host(c.ds_last)[:1], []
        for i in reversed(range(n)):
            r = start(i, s[i], ds)
            out.append([r[x][part(i)[1]] for x in NAMES[:5]])
            last = r["ds0"]
            ds = start(i, s[i], zero)["ds0"] if i == drop_back else last
        return dict(zip(NAMES, [np.concatenate(x) for x in zip(*out[::-1])]), ds0=last)

    want = joined()
    half = lambda x: HALF[c.io] if x in ("o", "dq", "dk", "dv") else HALF["f32"]   # noqa: E731
    # which joint is dropped, and which results have to notice
    if back:
        tries = [(dict(drop=0), ("dq", "dk", "dbeta")), (dict(drop=1), ("dq", "dk", "dbeta")), (dict(drop=n - 2), ("dq", "dk", "dbeta")),
                 (dict(drop_back=n - 1), ("dk", "dv", "ds0")), (dict(drop_back=n - 2), ("dk", "dv", "ds0")), (dict(drop_back=1), ("dk", "dv", "ds0"))]
    else:
        tries = [(dict(drop=0), ("o", "s_last")), (dict(drop=1), ("o", "s_last")), (dict(drop=n - 2), ("o", "s_last"))]
    for which, results in tries:
        other = joined(**which)
        for x in results:
            over = beyond(want[x], other[x], half(x), 2 if back else 1)
            assert over > 8, f"{which} would leave {x} at {over:.3g} of its bound"


CASES = [
    # dk, dv, io, decay
    (64, 64, "bf16", "token"),
    (64, 64, "f32", "token"),
    (128, 128, "bf16", "token"),
    (128, 128, "f32", "head"),
    (256, 256, "bf16", "token"),
    (256, 256, "f32", "token"),
    (33, 77, "bf16", "head"),
    (50, 130, "f32", "token"),
    (100, 40, "bf16", "token"),
    (127, 201, "f32", "token"),
    (130, 70, "bf16", "token"),
    (201, 33, "f32", "head"),
]


def make(dk, dv, io, decay):
    # the last sequence ends in a piece of one token, the one before has no token, the first has five pieces
    lens = [290, 64, 0, 193]
    seed = dk + dv
    return slow(Case(lens, 2, 1, dk, dv, io, decay, seed=seed), np.random.default_rng(seed))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_outputs_over_joints_that_count(case):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta fwd over joints {case}")
    c = make(*case)
    joints_count(c, 64, False)
    o, s = ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s0=c.s0, return_state=True, piece_len=64)
    torch.cuda.synchronize()
    check_fwd(c, o, s)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_gradients_over_joints_that_count(case):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta bwd over joints {case}")
    c = make(*case)
    joints_count(c, 64, True)
    r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=64)
    torch.cuda.synchronize()
    check_grads(c, r)
