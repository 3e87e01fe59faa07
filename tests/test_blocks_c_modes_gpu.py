"""GPU: the block operators' C entry points with the arguments that the binding's wrappers always
give left out: gradients without dg, with only one of the states, residual gradients in place,
left out, and without x.  What they give is bitwise what the full call gives (which
test_linattn_gpu.py and test_norms_gpu.py compare with float64)."""
import sys

import numpy as np
import pytest

import block_ref as ref
from test_linattn_bounds_gpu import near
from test_linattn_gpu import Case, check_grads

pytestmark = pytest.mark.gpu


def announce(msg):
    print(f"\n[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


NO_DG = [
    # lens, heads, kheads, dk, dv, io, state, piece, rows behind
    ([70, 1, 130], 2, 2, 64, 64, "bf16", True, 0, 5),
    ([70, 1, 130], 4, 2, 64, 64, "bf16", True, 64, 3),
    ([200], 3, 3, 33, 45, "bf16", False, 64, 0),
    ([200, 0, 9], 6, 2, 127, 40, "bf16", False, 64, 7),
    ([90, 40], 2, 2, 256, 200, "bf16", True, 64, 2),
    ([70, 33], 2, 2, 64, 96, "f32", True, 64, 5),
    ([70, 33], 4, 1, 31, 30, "f32", False, 0, 1),
    ([0, 0], 2, 2, 64, 64, "bf16", True, 0, 66),
    ([1, 0, 33, 64, 70] * 30, 6, 3, 128, 64, "bf16", True, 0, 0),
]


@pytest.mark.parametrize("case,packed", [(c, True) for c in NO_DG] + [(c, False) for c in NO_DG if len(c[0]) == 1],
                         ids=lambda c: "-".join(str(x).replace(" ", "")[:30] for x in c) if isinstance(c, tuple) else str(c))
def test_gradients_without_dg(case, packed):
    import torch
    import selective_state_space_79_amd as ssm

    lens, heads, kheads, dk, dv, io, state, piece, extra = case
    announce(f"no dg {case} packed {packed}")
    c = Case(lens, heads, kheads, dk, dv, io, "token", state, seed=dk, extra=extra if packed else 0)
    cu = c.cu if packed else None
    kw = dict(do=c.do, scale=c.scale, cu_seqlens=cu, s0=c.s0, ds_last=c.ds_last, piece_len=piece)
    want = ssm.linattn_bwd(c.q, c.k, c.v, c.g, **kw)
    got = {n: torch.full_like(t, 7.0) for n, t in want.items() if n != "dg"}
    dims = ssm.make_linattn_dims(c.T, c.n, heads, kheads, dk, dv, io_dtype=int(io == "bf16"), scale=c.scale, piece_len=piece,
                                 nslots=c.n)
    ws = torch.empty(ssm.ssm_linattn_bwd_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    dims.workspace, dims.workspace_bytes = ws.data_ptr(), ws.numel()
    grads = ssm.SsmLinattnGrads(*[got[n].data_ptr() if n in got else None for n in ("dq", "dk", "dv", "dg", "ds0")])
    st = ssm.ssm_linattn_bwd(c.q, c.k, c.v, c.g, cu, c.s0, c.do, c.ds_last, grads, dims)
    torch.cuda.synchronize()
    assert st == ssm.SSM_OK
    for n in got:
        assert torch.equal(got[n], want[n]), n
    if packed and extra:
        assert all(not got[n][int(c.starts[-1]):].any() for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("first,last", [(True, False), (False, True)])
@pytest.mark.parametrize("piece", [0, 64])
def test_gradients_with_one_of_the_states(first, last, piece, io):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"states {first} {last} piece {piece} {io}")
    c = Case([130, 0, 75], 4, 2, 64, 72, io, seed=50)
    zero = np.zeros_like(c.host(c.s0))
    s0, ds = (c.s0 if first else None), (c.ds_last if last else None)
    r = ssm.linattn_bwd(c.q, c.k, c.v, c.g, do=c.do, scale=c.scale, cu_seqlens=c.cu, s0=s0, ds_last=ds, piece_len=piece)
    torch.cuda.synchronize()
    if not first:
        c.s0 = None
    if not last:
        c.ds_last = None
    assert ("ds0" in r) == first
    check_grads(c, r)
    # a gradient of the starting state that C callers may ask for without one
    if not first:
        want = ref.linattn_grads(*(c.host(t) for t in (c.q, c.k, c.v)), c.gfull(), c.scale, c.starts, c.host(c.do), None,
                                 c.host(c.ds_last))["ds0"]
        terms = ref.linattn_grads(*(np.abs(c.host(t)) for t in (c.q, c.k, c.v)), c.gfull(), c.scale, c.starts,
                                  np.abs(c.host(c.do)), None, np.abs(c.host(c.ds_last)))["ds0"]
        dims = ssm.make_linattn_dims(c.T, c.n, 4, 2, 64, 72, io_dtype=int(io == "bf16"), scale=c.scale, piece_len=piece,
                                     nslots=c.n)
        ws = torch.empty(ssm.ssm_linattn_bwd_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
        dims.workspace, dims.workspace_bytes = ws.data_ptr(), ws.numel()
        got = {n: torch.full_like(r[n], 7.0) for n in ("dq", "dk", "dv", "dg")}
        ds0 = torch.full(zero.shape, 7.0, device="cuda")
        grads = ssm.SsmLinattnGrads(*[got[n].data_ptr() for n in ("dq", "dk", "dv", "dg")], ds0.data_ptr())
        assert ssm.ssm_linattn_bwd(c.q, c.k, c.v, c.g, c.cu, None, c.do, c.ds_last, grads, dims) == ssm.SSM_OK
        torch.cuda.synchronize()
        near("ds0", ds0, want, terms, "f32", 2.0 ** -14)
        assert all(torch.equal(got[n], r[n]) for n in got)


@pytest.mark.parametrize("io,res", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,dim", [(300, 256), (7, 1030), (3, 8200)])
def test_residual_gradients_in_place_left_out_and_without_x(rows, dim, io, res):
    import torch
    import selective_state_space_79_amd as ssm

    announce(f"residual gradients {rows}x{dim} {io} {res}")
    t = dict(bf16=torch.bfloat16, f32=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    x, dy, r, dr = rnd(rows, dim).to(t[io]), rnd(rows, dim).to(t[io]), rnd(rows, dim).to(t[res]), rnd(rows, dim).to(t[res])
    w, scale, post = rnd(dim), rnd(dim), rnd(dim)
    dims = ssm.SsmAddNormDims(rows, dim, 0, 0, 0, 0, int(io == "bf16"), int(res == "bf16"), 1e-5, 0, None, 0)
    ws = torch.empty(ssm.ssm_add_norm_bwd_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    dims.workspace, dims.workspace_bytes = ws.data_ptr(), ws.numel()
    for sc, po in ((scale, post), (scale, None), (None, post), (None, None)):
        want = ssm.add_norm_bwd(x, r, w, dy=dy, dr=dr, scale=sc, post_weight=po)
        for how in ("left out", "in place", "no x"):
            if how == "no x" and (sc is not None or po is not None):
                continue
            dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
            dsc, dpo = (None if s is None else torch.full_like(w, 7.0) for s in (sc, po))
            into = dr.clone()
            dres = into if how == "in place" else None
            st = ssm.ssm_add_norm_bwd(None if how == "no x" else x, r, sc, po, w, dy, into, dx, dres, dw, dsc, dpo, dims)
            torch.cuda.synchronize()
            assert st == ssm.SSM_OK
            assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dweight"]), how
            assert torch.equal(into, want["dresidual"] if how == "in place" else dr), how
            assert sc is None or torch.equal(dsc, want["dscale"])
            assert po is None or torch.equal(dpo, want["dpost_weight"])
