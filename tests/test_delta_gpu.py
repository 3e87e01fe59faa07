"""GPU parity of the gated delta rule (ssm_delta_fwd, _step, _bwd) against the float64 recurrence
of delta_ref.py.

Bounds.  With keys of length one, 0 <= beta <= 2 and decays of at most one no step makes a state,
or an error in one, longer, so what the roundings of each token leave adds up at most.  A token's
row passes sums of dk and of 64 terms, each term and each addition rounded by at most 2^-24 of the
sums' own size: up to 256 + 128 + 16 = 400 roundings.  Over 300 tokens that is 1.2e5 roundings of
random sign, whose sum is about their root times 2^-25: 346 * 2^-25 = 1e-5 < 2^-16 of the values'
norm.  So the error of an output or state stays below 2^-16 of the norm of its own head (NORM),
and a single value's, eight times its mean square at most, below 2^-13 of the head's largest
(ONE).  An output in bf16 is off by a further 2^-8 of its value.  Gradients pass the same sums
twice (states there, their gradients back): twice the bounds.
"""
import sys

import numpy as np
import pytest

import delta_ref as ref

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
NORM, ONE = 2.0 ** -16, 2.0 ** -13


def announce(msg):
    print(f"\n[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


def dtype(io):
    import torch

    return torch.bfloat16 if io == "bf16" else torch.float32


def unit(a):
    return a / np.sqrt((a * a).sum(-1, keepdims=True) + 1e-12)


class Case:
    """Seeded inputs of one call, on the device and as the float64 values they stand for."""

    def __init__(self, lens, heads, kheads, dk, dv, io="bf16", decay="token", state=True, seed=0, extra=0, gmin=1.6, top=1.9):
        import torch

        rng = np.random.default_rng(seed)
        self.lens, self.io, self.decay = lens, io, decay
        self.starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        self.T, self.n, self.scale = int(self.starts[-1]) + extra, len(lens), dk ** -0.5
        T = self.T
        put = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().to(dtype(io))   # noqa: E731
        self.q, self.k = put(unit(rng.standard_normal((T, kheads, dk)))), put(unit(rng.standard_normal((T, kheads, dk))) * 0.99)
        self.v, self.do = put(rng.standard_normal((T, heads, dv))), put(rng.standard_normal((T, heads, dv)))
        shape = (heads,) if decay == "head" else (T, heads)
        self.g = torch.from_numpy((-np.exp(rng.uniform(np.log(1e-3), np.log(gmin), shape))).astype(np.float32)).cuda()
        self.beta = torch.from_numpy(rng.uniform(0, top, (T, heads)).astype(np.float32)).cuda()
        f32 = lambda: torch.from_numpy(rng.standard_normal((self.n, heads, dk, dv)).astype(np.float32)).cuda()  # noqa: E731
        self.s0 = f32() if state else None
        self.ds_last = f32() if state else None
        self.cu = torch.from_numpy(self.starts.astype(np.int32)).cuda()

    def rows(self):
        return self.q, self.k, self.v, self.g, self.beta

    def host(self, t):
        return None if t is None else t.double().cpu().numpy()

    def args(self):
        g = self.host(self.g)
        g = np.broadcast_to(g, (self.T, g.shape[-1])) if g.ndim == 1 else g
        return self.host(self.q), self.host(self.k), self.host(self.v), g, self.host(self.beta), self.scale, self.starts

    def ref_fwd(self):
        return ref.delta(*self.args(), self.host(self.s0))

    def ref_bwd(self):
        return ref.delta_grads(*self.args(), self.host(self.do), self.host(self.s0), self.host(self.ds_last))


def check(name, got, want, io, heads_at=1, times=1, least=1e-30):
    """Head by head (axis heads_at): each value's error and the norm of all; `least` is allowed anyhow."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{name}: not finite"
    other = tuple(i for i in range(want.ndim) if i != heads_at)
    err, half = np.abs(got - want), HALF[io] * np.abs(want)
    rest = np.maximum(err - half, 0)
    big = np.abs(want).max(other, keepdims=True, initial=0)
    over = rest / (times * ONE * big + least)
    assert over.max(initial=0) <= 1, f"{name}: {over.max():.3g} of the bound at {np.unravel_index(over.argmax(), over.shape)}"
    a, b = np.sqrt((rest ** 2).sum(other)), np.sqrt((want ** 2).sum(other))
    a = a / (times * NORM * b + least * np.sqrt(want.size))
    assert (a <= 1).all(), f"{name}: {a.max():.3g} of the norm's bound"


def check_fwd(c, o, s_last=None):
    ro, rs = c.ref_fwd()
    n = int(c.starts[-1])
    check("o", o[:n], ro[:n], c.io)
    if s_last is not None:
        check("s_last", s_last, rs, "f32")


def check_grads(c, r):
    want = c.ref_bwd()
    n = int(c.starts[-1])
    for name in ("dq", "dk", "dv"):
        # a step of zero counts as 2^-64 in dk = dS u - S dr: |u| and |dr| are 2^-64 of |r| and |dS k|
        # at most, and rows and columns of states and their gradients stay under 2^10 here: 2^-43 in all
        check(name, r[name][:n], want[name][:n], c.io, times=2, least=2.0 ** -43 if name == "dk" else 1e-30)
    if c.decay == "head":
        # the head's sum over T tokens may cancel.  Errors e_t of norm 2 NORM |dg| at most have a sum
        # of sqrt(T) times that at most (Cauchy and Schwarz), whatever the sum of dg itself is
        n0 = int(c.starts[0])
        room = 2 * NORM * np.sqrt(n - n0) * np.sqrt((want["dg"] ** 2).sum(0))
        err = np.abs(c.host(r["dg"]) - want["dg"].sum(0))
        assert (err <= room + 1e-30).all(), f"dg: {(err / room).max():.3g} of the bound"
    else:
        check("dg", r["dg"][:n], want["dg"][:n], "f32", times=2)
    check("dbeta", r["dbeta"][:n], want["dbeta"][:n], "f32", times=2)
    if c.s0 is not None:
        check("ds0", r["ds0"], want["ds0"], "f32", times=2)


CASES = [
    # lens, heads, kheads, dk, dv, io, decay, state, piece
    ([1], 1, 1, 1, 1, "bf16", "token", True, 0),
    ([64], 2, 2, 64, 64, "bf16", "token", False, 0),
    ([65], 2, 1, 64, 128, "bf16", "token", True, 0),
    ([130], 3, 3, 128, 128, "bf16", "head", True, 0),
    ([1, 0, 31, 32, 33, 63, 64, 200], 4, 2, 128, 64, "bf16", "token", True, 0),
    ([300], 2, 2, 128, 128, "bf16", "token", True, 64),
    ([1, 0, 257, 64, 128], 2, 1, 128, 96, "bf16", "token", True, 128),
    ([150, 30], 2, 2, 256, 256, "bf16", "token", True, 64),
    ([90, 30], 2, 1, 256, 100, "bf16", "head", True, 0),
    ([70, 100], 3, 3, 40, 200, "bf16", "token", False, 64),
    ([100, 7], 3, 1, 33, 70, "bf16", "token", True, 0),
    ([200], 2, 1, 33, 77, "bf16", "token", True, 64),
    ([90], 2, 2, 200, 136, "bf16", "head", True, 0),
    ([1], 1, 1, 3, 5, "f32", "token", True, 0),
    ([64, 65], 2, 2, 64, 64, "f32", "token", True, 0),
    ([1, 77, 130], 6, 3, 72, 40, "f32", "token", True, 64),
    ([100], 2, 1, 128, 128, "f32", "token", False, 0),
    ([100, 40], 2, 2, 64, 128, "f32", "head", True, 64),
    ([140], 1, 1, 256, 250, "f32", "token", True, 64),
]
IDS = ["-".join(str(x).replace(" ", "") for x in c) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_matches_recurrence(case):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta fwd {case}")
    *a, piece = case
    c = Case(*a, seed=len(str(case)))
    o, s = ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s0=c.s0, return_state=True, piece_len=piece)
    torch.cuda.synchronize()
    check_fwd(c, o, s)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradients_match_recurrence(case):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta bwd {case}")
    *a, piece = case
    c = Case(*a, seed=len(str(case)))
    r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
    torch.cuda.synchronize()
    check_grads(c, r)


@pytest.mark.parametrize("heads,kheads,dk,dv", [(1, 1, 1, 1), (4, 2, 128, 128), (6, 3, 33, 77), (2, 1, 256, 256), (3, 3, 200, 15),
                                                (32, 16, 128, 128)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_step_matches_recurrence(io, heads, kheads, dk, dv):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta step {io} {heads} {kheads} {dk} {dv}")
    for batch in (1, 5, 70):
        for decay in ("token", "head"):
            c = Case([1] * batch, heads, kheads, dk, dv, io, decay, seed=batch)
            gen = torch.Generator().manual_seed(batch)
            slots = torch.randperm(batch + 3, generator=gen)[:batch].to(torch.int32).cuda()
            pool = torch.full((batch + 3, heads, dk, dv), 7.0, device="cuda")
            pool[slots.long()] = c.s0
            o = ssm.delta_step(*c.rows(), pool, slots=slots, scale=c.scale)
            torch.cuda.synchronize()
            check_fwd(c, o, pool[slots.long()])
            rest = [i for i in range(batch + 3) if i not in slots.tolist()]
            assert (pool[rest] == 7.0).all()


def test_steps_continue_a_prompt():
    """A prompt and single tokens after it: the whole sequence's results."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta prompt then steps")
    for io in ("bf16", "f32"):
        c = Case([40, 40], 4, 2, 64, 96, io, seed=3)
        ro, rs = c.ref_fwd()
        cut = 33
        at = lambda t, i: t.view(2, 40, *t.shape[1:])[:, i]      # noqa: E731
        head = [at(t, slice(0, cut)).contiguous() for t in c.rows()]
        o, s = ssm.delta_fwd(*head, scale=c.scale, s0=c.s0, return_state=True)
        check("o", o, ro.reshape(2, 40, 4, 96)[:, :cut], io, heads_at=2)
        for t in range(cut, 40):
            o = ssm.delta_step(*[at(x, t).contiguous() for x in c.rows()], s, scale=c.scale)
            check("o", o, ro.reshape(2, 40, 4, 96)[:, t], io)
        check("state", s, rs, "f32")


def test_forward_skips_padding_and_repeated_slots():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta slots")
    c = Case([50, 3, 70, 20, 40], 2, 1, 64, 64, seed=4)
    pool = torch.randn(6, 2, 64, 64, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    slots = torch.tensor([4, -1, 2, 4, 9], dtype=torch.int32, device="cuda")     # padding, repeated, out of range
    for piece in (0, 64):
        p, out = pool.clone(), torch.full_like(c.v, 5.0)
        ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s0=p, s_last=p, slots=slots, out=out, piece_len=piece)
        torch.cuda.synchronize()
        full = torch.zeros(5, 2, 64, 64, device="cuda")
        full[0], full[2] = pool[4], pool[2]
        ro, rs = ref.delta(*c.args(), c.host(full))
        for s, slot in ((0, 4), (2, 2)):
            a, b = c.starts[s], c.starts[s + 1]
            check("o", out[a:b], ro[a:b], "bf16")
            check("state", p[slot][None], rs[s][None], "f32")
        for s in (1, 3, 4):
            assert (out[c.starts[s]:c.starts[s + 1]] == 5.0).all()
        for i in (0, 1, 3, 5):
            assert torch.equal(p[i], pool[i])
    one = [t[:5].contiguous() for t in c.rows()]
    p, out = pool.clone(), torch.full_like(c.v[:5], 5.0)
    ssm.delta_step(*one, p, slots=slots, scale=c.scale, out=out)
    torch.cuda.synchronize()
    assert (out[[1, 3, 4]] == 5.0).all() and not (out[[0, 2]] == 5.0).all(-1).any()
    assert all(torch.equal(p[i], pool[i]) for i in (0, 1, 3, 5)) and not torch.equal(p[4], pool[4])


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_columns_of_one_projection(io, pad):
    """q, k, v, do and o as columns of wider buffers, packed or (batch, L): bitwise the packed results."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta columns {io} {pad}")
    B, L, H, Hk, dk, dv = 2, 75, 4, 2, 64, 64
    c = Case([L] * B, H, Hk, dk, dv, io, seed=pad)
    wide = 2 * Hk * dk + 2 * H * dv + pad
    buf = torch.zeros(B * L, wide, dtype=dtype(io), device="cuda")
    at, cols = 0, []
    for t in (c.q, c.k, c.v, c.do):
        n = t.shape[1] * t.shape[2]
        buf[:, at:at + n] = t.flatten(1)
        cols.append(buf[:, at:at + n].unflatten(-1, t.shape[1:]))
        at += n
    q, k, v, do = cols
    kw = dict(scale=c.scale, s0=c.s0)
    want, ws = ssm.delta_fwd(*c.rows(), cu_seqlens=c.cu, return_state=True, **kw)
    grads = ssm.delta_bwd(*c.rows(), do=c.do, cu_seqlens=c.cu, ds_last=c.ds_last, **kw)
    room = torch.zeros(B * L, H * dv + pad + 3, dtype=dtype(io), device="cuda")
    out = room[:, :H * dv].unflatten(-1, (H, dv))
    o, s = ssm.delta_fwd(q, k, v, c.g, c.beta, cu_seqlens=c.cu, return_state=True, out=out, **kw)
    assert torch.equal(o, want) and torch.equal(s, ws) and (room[:, H * dv:] == 0).all()
    r = ssm.delta_bwd(q, k, v, c.g, c.beta, do=do, cu_seqlens=c.cu, ds_last=c.ds_last, **kw)
    assert all(torch.equal(r[n], grads[n]) for n in grads)
    four = lambda t: t.unflatten(0, (B, L))     # noqa: E731
    o, s = ssm.delta_fwd(four(q), four(k), four(v), four(c.g), four(c.beta), return_state=True, **kw)
    assert torch.equal(o.flatten(0, 1), want) and torch.equal(s, ws)
    r = ssm.delta_bwd(four(q), four(k), four(v), four(c.g), four(c.beta), do=four(do), ds_last=c.ds_last, **kw)
    assert all(torch.equal(r[n].reshape(grads[n].shape), grads[n]) for n in grads)
    pool, pool2 = c.s0.clone(), c.s0.clone()
    a = ssm.delta_step(q[:2], k[:2], v[:2], c.g[:2], c.beta[:2], pool)
    b = ssm.delta_step(c.q[:2], c.k[:2], c.v[:2], c.g[:2], c.beta[:2], pool2)
    assert torch.equal(a, b) and torch.equal(pool, pool2)


def test_rows_behind_the_last_sequence():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta rows of no sequence")
    for io, piece in (("bf16", 0), ("bf16", 64), ("f32", 0)):
        c = Case([20, 100], 4, 2, 64, 64, io, seed=5, extra=30)
        c.cu += 7                                    # rows before the first sequence as well
        c.starts = c.starts + 7
        for t in c.rows()[:3] + (c.do,):
            t[:7] = float("nan")
            t[127:] = float("nan")
        for t in (c.g, c.beta):
            t[:7] = float("nan")
            t[127:] = float("nan")
        out = torch.full_like(c.v, 3.0)
        _, s = ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s0=c.s0, return_state=True, out=out, piece_len=piece)
        r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
        torch.cuda.synchronize()
        assert (out[:7] == 3.0).all() and (out[127:] == 3.0).all()
        ro, rs = ref.delta(*[np.nan_to_num(x) if isinstance(x, np.ndarray) else x for x in c.args()], c.host(c.s0))
        check("o", out[7:127], ro[7:127], io)
        check("s_last", s, rs, "f32")
        assert torch.isfinite(r["ds0"]).all()
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert (r[n][:7] == 0).all() and (r[n][127:] == 0).all() and torch.isfinite(r[n]).all(), n


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decays_and_steps_at_their_ends(io):
    """Decays of one and of zero (-inf, -200), steps of zero, one and two; nothing but a step of
    zero leaves the state to its decay."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta ends {io}")
    c = Case([150, 40], 3, 3, 64, 64, io, seed=6)
    c.k = c.k / c.k.float().norm(dim=-1, keepdim=True).to(c.k.dtype) * 0.99
    c.g[:, 0] = 0.0
    c.g[20, 1], c.g[77, 1], c.g[64, 2] = float("-inf"), -200.0, -1e30
    c.beta[:, 0] = 0.0
    c.beta[30:60, 1] = 0.0
    c.beta[::3, 2], c.beta[1::3, 2] = 1.0, 2.0
    for piece in (0, 64):
        o, s = ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s0=c.s0, return_state=True, piece_len=piece)
        r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
        torch.cuda.synchronize()
        check_fwd(c, o, s)
        check_grads(c, r)
        assert torch.equal(s[:, 0], c.s0[:, 0])                # no decay, no step
        assert (r["dv"][:, 0] == 0).all()


def test_bad_values_stay_in_their_sequence():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta bad values")
    for bad in (float("nan"), float("inf")):
        for io in ("bf16", "f32"):
            c = Case([50, 60, 40], 2, 1, 64, 64, io, seed=7)
            good = Case([50, 60, 40], 2, 1, 64, 64, io, seed=7)
            for t in c.rows()[:3] + (c.do, c.g, c.beta):
                t[50:110] = bad
            c.s0[1] = bad
            c.ds_last[1] = bad
            kw = dict(scale=c.scale, cu_seqlens=c.cu)
            o, s = ssm.delta_fwd(*c.rows(), s0=c.s0, return_state=True, **kw)
            r = ssm.delta_bwd(*c.rows(), do=c.do, s0=c.s0, ds_last=c.ds_last, **kw)
            wo, wss = ssm.delta_fwd(*good.rows(), s0=good.s0, return_state=True, **kw)
            wr = ssm.delta_bwd(*good.rows(), do=good.do, s0=good.s0, ds_last=good.ds_last, **kw)
            for a, b in ((o, wo), *((r[n], wr[n]) for n in ("dq", "dk", "dv", "dg", "dbeta"))):
                assert torch.equal(a[:50], b[:50]) and torch.equal(a[110:], b[110:])
            for a, b in ((s, wss), (r["ds0"], wr["ds0"])):
                assert torch.equal(a[[0, 2]], b[[0, 2]])


def test_repeated_calls_are_bitwise_equal():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta repeated")
    for decay in ("token", "head"):
        c = Case([700, 90, 1], 4, 1, 128, 128, decay=decay, seed=8)
        kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0)
        first = None
        for _ in range(3):
            o, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
            r = [o, s, *ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw).values()]
            first = first or r
            assert all(torch.equal(a, b) for a, b in zip(r, first))


def test_gradients_against_differences():
    """Directional derivatives of the float64 recurrence by central differences: an error of h^2
    (1e-8 of values near one, with room for third derivatives) and 1e-16 / h in rounding."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta differences")
    c = Case([37, 5], 2, 1, 24, 40, "f32", seed=9, gmin=0.3)
    r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last)
    torch.cuda.synchronize()
    q, k, v, g, beta, scale, starts = c.args()
    s0, do, dsl = c.host(c.s0), c.host(c.do), c.host(c.ds_last)
    rng = np.random.default_rng(1)

    def loss(**d):
        a = dict(q=q, k=k, v=v, g=g, beta=beta, s0=s0)
        for n, x in d.items():
            a[n] = a[n] + x
        o, last = ref.delta(a["q"], a["k"], a["v"], a["g"], a["beta"], scale, starts, a["s0"])
        return (o * do).sum() + (last * dsl).sum()

    h = 1e-4
    for name, base in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("s0", s0)):
        way = rng.standard_normal(base.shape)
        want = (loss(**{name: h * way}) - loss(**{name: -h * way})) / (2 * h)
        got = (c.host(r["d" + name]) * way).sum()
        size = np.sqrt((c.host(r["d" + name]) ** 2).sum()) * np.sqrt((way ** 2).sum())
        assert abs(got - want) <= (2 * NORM + 1e-6) * size, (name, got, want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_what_is_written_twice_is_taken_back(io):
    """One key and one value again and again, step one, no decay: after the first token the state
    is k v^T, and what each next one lacks is zero up to rounding.  The key has one nonzero
    entry, so sums have one term: v and its parts' products are rounded a few times a token,
    under 8 * 2^-24 of v, and 200 tokens' of random sign to 15 times 2^-24 * 8 < 2^-17."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta taken back {io}")
    T, H, d = 200, 2, 64
    rng = np.random.default_rng(2)
    k = torch.zeros(T, H, d)
    k[:, 0, 5], k[:, 1, 63] = 1.0, -1.0
    v = torch.from_numpy(rng.standard_normal((1, H, d)).astype(np.float32)).expand(T, H, d).contiguous()
    k, v = k.cuda().to(dtype(io)), v.cuda().to(dtype(io))
    g, beta = torch.zeros(T, H, device="cuda"), torch.ones(T, H, device="cuda")
    for piece in (0, 64):
        o, s = ssm.delta_fwd(k, k, v, g, beta, return_state=True, piece_len=piece)
        torch.cuda.synchronize()
        want = torch.zeros(1, H, d, d, dtype=torch.float64)
        want[0, 0, 5], want[0, 1, 63] = v[0, 0].double().cpu(), -v[0, 1].double().cpu()
        assert ((s.double().cpu() - want).abs() <= 2.0 ** -17 * v.double().abs().cpu().max()).all()
        assert ((o.double() - v.double()).abs() <= (HALF[io] + 2.0 ** -17) * v.double().abs().max()).all()


def test_other_streams_and_captured_calls():
    """On a stream of its own, and captured into two graphs that live beside eager calls: each
    replay gives the eager results, with new inputs copied in between."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta streams and graphs")
    c = Case([300, 40, 1], 4, 2, 64, 64, seed=10)
    d = Case([300, 40, 1], 4, 2, 64, 64, seed=11)
    kw = dict(scale=c.scale, cu_seqlens=c.cu, piece_len=64)

    def calls(x, stream=None):
        o, s = ssm.delta_fwd(*x.rows(), s0=x.s0, return_state=True, stream=stream, **kw)
        r = ssm.delta_bwd(*x.rows(), do=x.do, s0=x.s0, ds_last=x.ds_last, stream=stream, **kw)
        pool = x.s0.clone()
        one = [t[:3].contiguous() for t in x.rows()]
        return [o, s, *r.values(), ssm.delta_step(*one, pool, scale=c.scale, stream=stream), pool]

    want = [[t.clone() for t in calls(x)] for x in (c, d)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls(c)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs = []
    for x in (c, d):
        with torch.cuda.stream(side):
            calls(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = calls(x)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), w in zip(graphs, want):
            for t in out[:-1]:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, w))
            again = calls(c)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(again, want[0]))
    keep = c.v.clone()
    c.v.copy_(d.v)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    fresh = calls(c)
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], fresh))
    c.v.copy_(keep)


def test_two_calls_at_once():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta two streams")
    sets = [Case([400, 100], 4, 2, 64, 128, seed=12), Case([333], 2, 2, 128, 64, seed=13)]

    def calls(c, stream=None):
        kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0, stream=stream)
        o, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
        return [o, s, *ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw).values()]

    want = [calls(c) for c in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, c in enumerate(sets):
            got[i].append(calls(c, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_random_shapes():
    import torch
    import selective_state_space_79_amd as ssm

    rng = np.random.default_rng(14)
    for i in range(24):
        kheads = int(rng.choice([1, 2, 3]))
        heads = kheads * int(rng.choice([1, 2, 4]))
        dk, dv = int(rng.integers(1, 257)), int(rng.integers(1, 257))
        lens = [int(x) for x in rng.integers(0, 130, int(rng.integers(1, 5)))]
        if sum(lens) == 0:
            lens = [1]
        io, piece = str(rng.choice(["bf16", "f32"])), int(rng.choice([0, 64, 128]))
        decay, state = str(rng.choice(["token", "head"])), bool(rng.random() < 0.7)
        announce(f"delta random {i}: {lens} {heads} {kheads} {dk} {dv} {io} {decay} {state} {piece}")
        c = Case(lens, heads, kheads, dk, dv, io, decay, state, seed=i)
        kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0, piece_len=piece)
        o, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
        r = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw)
        torch.cuda.synchronize()
        check_fwd(c, o, s)
        check_grads(c, r)


def test_pieces_by_the_library_choice():
    """Long enough sequences that the library cuts them itself: the forced pieces' results up to
    rounding, and those of one piece."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta pieces of the library's choice")
    for lens in ([3000], [1500, 1500], [2500, 7, 1, 0, 400]):
        c = Case(lens, 1, 1, 64, 64, seed=len(lens))
        kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0)
        whole, sw = ssm.delta_fwd(*c.rows(), return_state=True, piece_len=1 << 20, **kw)
        gw = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, piece_len=1 << 20, **kw)
        o, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
        g = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw)
        torch.cuda.synchronize()
        check("o", o, c.host(whole), "bf16")
        check("s", s, c.host(sw), "f32")
        for n in gw:
            check(n, g[n], c.host(gw[n]), "bf16" if n in ("dq", "dk", "dv") else "f32", times=2)


def test_many_short_sequences():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta many short sequences")
    rng = np.random.default_rng(15)
    lens = [int(x) for x in rng.integers(0, 5, 700)]
    c = Case(lens, 2, 1, 16, 24, seed=15)
    kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0)
    o, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
    r = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw)
    torch.cuda.synchronize()
    check_fwd(c, o, s)
    check_grads(c, r)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("heads,kheads,dk,dv", [(6, 2, 40, 24), (8, 2, 128, 33), (4, 2, 200, 64)])
def test_shared_heads_of_many_chunks(heads, kheads, dk, dv, decay, io):
    """Enough chunks that the heads which share q and k go one after the other in the gradients."""
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"delta shared heads of many chunks {heads} {kheads} {dk} {dv} {decay} {io}")
    rng = np.random.default_rng(21)
    lens = [70, 0, 33] + [int(x) for x in rng.integers(0, 3, 600)]
    c = Case(lens, heads, kheads, dk, dv, io, decay, seed=heads)
    r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last)
    again = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=c.s0, ds_last=c.ds_last)
    torch.cuda.synchronize()
    check_grads(c, r)
    assert all(torch.equal(r[n], again[n]) for n in r)


def test_offsets_past_32_bits():
    """Rows and states behind the first 2^31 elements: bitwise the results of a call of their own."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta past 32 bits")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    c = Case([100, 50], 2, 1, 64, 64, seed=16)
    T, row = 70000, 32768
    buf = torch.zeros(T, row, dtype=torch.bfloat16, device="cuda")
    assert buf.numel() > 1 << 31
    cols, at = [], row - 512
    for t in (c.q, c.k, c.v, c.do):
        n = t.shape[1] * t.shape[2]
        buf[T - 150:, at:at + n] = t.flatten(1)
        cols.append(buf[:, at:at + n].unflatten(-1, t.shape[1:]))
        at += n
    q, k, v, do = cols
    g, beta = torch.zeros(T, 2, device="cuda"), torch.zeros(T, 2, device="cuda")
    g[T - 150:], beta[T - 150:] = c.g, c.beta
    cu = c.cu + (T - 150)
    room = torch.full((T, row), 2.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, 64:192].unflatten(-1, (2, 64))
    kw = dict(scale=c.scale, s0=c.s0)
    want, sw = ssm.delta_fwd(*c.rows(), cu_seqlens=c.cu, return_state=True, **kw)
    _, s = ssm.delta_fwd(q, k, v, g, beta, cu_seqlens=cu, return_state=True, out=out, **kw)
    assert torch.equal(out[T - 150:], want) and torch.equal(s, sw) and (room[:T - 150] == 2.0).all()
    gw = ssm.delta_bwd(*c.rows(), do=c.do, cu_seqlens=c.cu, ds_last=c.ds_last, **kw)
    r = ssm.delta_bwd(q, k, v, g, beta, do=do, cu_seqlens=cu, ds_last=c.ds_last, **kw)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(r[n][T - 150:], gw[n]) and (r[n][:T - 150] == 0).all(), n
    assert torch.equal(r["ds0"], gw["ds0"])
    del buf, room, out, cols, q, k, v, do
    pool = torch.zeros(1100, 32, 256, 256, device="cuda")
    assert pool.numel() > 1 << 31
    d = Case([1, 1], 32, 16, 256, 256, seed=17)
    pool[1098:] = d.s0
    slots = torch.tensor([1098, 1099], dtype=torch.int32, device="cuda")
    few = d.s0.clone()
    a = ssm.delta_step(*d.rows(), pool, slots=slots, scale=d.scale)
    b = ssm.delta_step(*d.rows(), few, scale=d.scale)
    assert torch.equal(a, b) and torch.equal(pool[1098:], few) and (pool[:1098] == 0).all()


def test_empty_sequences_keep_their_states():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta empty sequences")
    c = Case([0, 40, 0, 0], 2, 1, 32, 48, seed=18)
    kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0)
    _, s = ssm.delta_fwd(*c.rows(), return_state=True, **kw)
    r = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw)
    torch.cuda.synchronize()
    for i in (0, 2, 3):
        assert torch.equal(s[i], c.s0[i]) and torch.equal(r["ds0"][i], c.ds_last[i])


def test_nothing_but_empty_sequences():
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta nothing but empty sequences")
    for io in ("bf16", "f32"):
        for piece in (0, 64):
            c = Case([0, 0, 0], 2, 1, 40, 48, io, seed=22, extra=300)
            kw = dict(scale=c.scale, cu_seqlens=c.cu, s0=c.s0, piece_len=piece)
            out = torch.full_like(c.v, 3.0)
            _, s = ssm.delta_fwd(*c.rows(), return_state=True, out=out, **kw)
            r = ssm.delta_bwd(*c.rows(), do=c.do, ds_last=c.ds_last, **kw)
            torch.cuda.synchronize()
            assert torch.equal(s, c.s0) and torch.equal(r["ds0"], c.ds_last) and (out == 3.0).all()
            assert all((r[n] == 0).all() for n in ("dq", "dk", "dv", "dg", "dbeta"))


def test_states_into_slots_from_zeros():
    """No starting states, final ones into a pool by slots; gradients without states of any kind,
    and through the C call with ds0 though there is no s0."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("delta states into slots")
    c = Case([70, 33], 4, 2, 64, 64, state=False, seed=23)
    for piece in (0, 64):
        pool = torch.full((5, 4, 64, 64), 7.0, device="cuda")
        slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
        o = ssm.delta_fwd(*c.rows(), scale=c.scale, cu_seqlens=c.cu, s_last=pool, slots=slots, piece_len=piece)
        torch.cuda.synchronize()
        check_fwd(c, o, pool[[3, 1]])
        assert (pool[[0, 2, 4]] == 7.0).all()
        r = ssm.delta_bwd(*c.rows(), do=c.do, scale=c.scale, cu_seqlens=c.cu, piece_len=piece)
        check_grads(c, r)
        assert "ds0" not in r
        dims = ssm.make_linattn_dims(tokens=103, nseq=2, nheads=4, kheads=2, dk=64, dv=64, scale=c.scale, piece_len=piece)
        ws = torch.empty(ssm.ssm_delta_bwd_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
        dims.workspace, dims.workspace_bytes = ws.data_ptr(), ws.numel()
        g = {n: torch.full_like(r[n], 5.0) for n in ("dq", "dk", "dv", "dg", "dbeta")}
        ds0 = torch.full((2, 4, 64, 64), 5.0, device="cuda")
        grads = ssm.SsmDeltaGrads(*[g[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dbeta")], ds0.data_ptr())
        assert ssm.ssm_delta_bwd(*c.rows(), c.cu, None, c.do, None, grads, dims, None) == ssm.SSM_OK
        torch.cuda.synchronize()
        assert all(torch.equal(g[n], r[n]) for n in g)
        check("ds0", ds0, c.ref_bwd()["ds0"], "f32", times=2)


def test_refused_calls():
    import torch
    import selective_state_space_79_amd as ssm

    c = Case([20], 2, 1, 16, 16, seed=19)
    q, k, v, g, beta = c.rows()
    with pytest.raises(ValueError, match="beta"):
        ssm.delta_fwd(q, k, v, g, beta[:5])
    with pytest.raises(TypeError, match="beta"):
        ssm.delta_fwd(q, k, v, g, beta.double())
    with pytest.raises(ValueError, match="overlap"):
        ssm.delta_fwd(q, k, v[:1].expand(20, 2, 16), g, beta)
    with pytest.raises(ssm.SsmError):
        ssm.delta_fwd(q, k, v, g, beta, out=v)
    with pytest.raises(ssm.SsmError):
        ssm.delta_fwd(q, k, v, g, beta, piece_len=32)
    with pytest.raises(ValueError, match="do"):
        ssm.delta_bwd(q, k, v, g, beta, do=c.do[:3])
    with pytest.raises(ValueError, match="states"):
        ssm.delta_step(q, k, v, g, beta, c.s0[:, :1])


def test_a_block_with_its_norms():
    """A layer norm, projections, keys and queries of length one, the mixer, the gated norm behind
    it and the way back, against the same block in float64 with torch's own derivatives."""
    import torch
    import selective_state_space_79_amd as ssm

    announce("a delta block")
    gen = torch.Generator().manual_seed(20)
    T, D, H, Hk, d = 90, 128, 4, 2, 32
    cu = torch.tensor([0, 33, 90], dtype=torch.int32)
    rand = lambda *s, m=1.0: torch.randn(*s, generator=gen, dtype=torch.float64) * m   # noqa: E731
    x, w1, b1, w2 = rand(T, D) + 0.5, 1 + rand(D, m=0.1), rand(D, m=0.1), 1 + rand(d, m=0.1)
    W = {n: rand(D, h * d, m=D ** -0.5) for n, h in (("q", Hk), ("k", Hk), ("v", H), ("z", H))}
    Wg, Wb, top = rand(D, H, m=D ** -0.5), rand(D, H, m=D ** -0.5), rand(T, H * d)
    names = ["x", "w1", "b1", "w2", *W]
    leaf = {n: t.float().double().requires_grad_() for n, t in dict(x=x, w1=w1, b1=b1, w2=w2, **W).items()}
    Wg, Wb, top = Wg.float().double(), Wb.float().double(), top.float().double()

    def plain():
        p = leaf
        c = p["x"] - p["x"].mean(-1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * p["w1"] + p["b1"]
        n = lambda t: t / torch.sqrt((t * t).sum(-1, keepdim=True) + d * 1e-5)   # noqa: E731
        q, k = (n((y @ p[i]).view(T, Hk, d)).repeat_interleave(H // Hk, 1) for i in "qk")
        v, z = (y @ p["v"]).view(T, H, d), (y @ p["z"]).view(T, H, d)
        a, beta = torch.exp(-torch.nn.functional.softplus(y @ Wg)), torch.sigmoid(y @ Wb)
        rows = []
        for s in range(2):
            S = torch.zeros(H, d, d, dtype=torch.float64)
            for t in range(cu[s], cu[s + 1]):
                S = S * a[t][:, None, None]
                r = v[t] - (S * k[t][:, :, None]).sum(1)
                S = S + k[t][:, :, None] * (beta[t][:, None] * r)[:, None, :]
                rows.append(d ** -0.5 * (S * q[t][:, :, None]).sum(1))
        o = torch.stack(rows)
        h = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-5) * p["w2"] * torch.nn.functional.silu(z)
        return h.reshape(T, -1)

    want = plain()
    (want * top).sum().backward()
    g = {n: t.detach().float().cuda() for n, t in leaf.items()}
    cud, topd = cu.cuda(), top.float().cuda()
    y = ssm.layer_norm_fwd(g["x"], g["w1"], g["b1"])
    pq, pk, pv, pz = (y @ g[i] for i in "qkvz")
    ones = torch.full((d,), d ** -0.5, device="cuda")
    q, k = (ssm.gated_norm_fwd(t, None, ones, group_size=d).view(T, Hk, d) for t in (pq, pk))
    fg, fb = y @ Wg.float().cuda(), y @ Wb.float().cuda()
    dec, beta = -torch.nn.functional.softplus(fg), torch.sigmoid(fb)
    v = pv.view(T, H, d)
    o = ssm.delta_fwd(q, k, v, dec, beta, scale=d ** -0.5, cu_seqlens=cud)
    h = ssm.gated_norm_fwd(o.view(T, -1), pz, g["w2"], group_size=d, gate_first=False)
    near = lambda n, a, b, tol: (a.double().cpu() - b).norm() <= tol * b.norm() or pytest.fail(   # noqa: E731
        f"{n}: {float((a.double().cpu() - b).norm() / b.norm()):.3g}")
    near("h", h, want.detach(), 2 * NORM)
    bn = ssm.gated_norm_bwd(o.view(T, -1), pz, g["w2"], dy=topd, group_size=d, gate_first=False)
    bd = ssm.delta_bwd(q, k, v, dec, beta, do=bn["dx"].view(T, H, d), scale=d ** -0.5, cu_seqlens=cud)
    dpq, dpk = (ssm.gated_norm_bwd(t, None, ones, dy=bd[n].reshape(T, -1), group_size=d)["dx"] for t, n in ((pq, "dq"), (pk, "dk")))
    dg, db = -bd["dg"] * torch.sigmoid(fg), bd["dbeta"] * beta * (1 - beta)
    dpv = bd["dv"].reshape(T, -1)
    dy = dpq @ g["q"].T + dpk @ g["k"].T + dpv @ g["v"].T + bn["dz"] @ g["z"].T + dg @ Wg.float().cuda().T + db @ Wb.float().cuda().T
    bl = ssm.layer_norm_bwd(g["x"], g["w1"], dy=dy)
    got = dict(x=bl["dx"], w1=bl["dweight"], b1=bl["dbias"], w2=bn["dweight"], q=y.T @ dpq, k=y.T @ dpk, v=y.T @ dpv, z=y.T @ bn["dz"])
    for n in names:
        near(n, got[n], leaf[n].grad, 8 * NORM)      # four operators in a row, twice the bound each
