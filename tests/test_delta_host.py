"""Host-side checks of the gated delta rule and of the layer norm that need no GPU: every refusal
is returned before anything reaches the HIP runtime (fake addresses, never dereferenced); the
binding's own checks raise on the CPU."""
import pytest

import selective_state_space_79_amd as ssm
from test_blocks_host import at, call, lin, with_workspace

FWD = ["q", "k", "v", "g", "beta", "-cu", "-slots", "-s0", "o", "-s_last"]
STEP = ["q", "k", "v", "g", "beta", "-slots", "states", "o"]
BWD = ["q", "k", "v", "g", "beta", "-cu", "-s0", "do", "-ds_last"]
LAYER = ["x", "w", "-b", "y"]
LAYER_B = ["x", "w", "dy", "dx", "dw", "-db"]


def ready(**kw):
    """Dims with a workspace of the size that the forward asks for."""
    d = lin(**kw)
    return with_workspace(d, ssm.ssm_delta_fwd_workspace_bytes(d))


def ready_b(**kw):
    d = lin(**kw)
    return with_workspace(d, ssm.ssm_delta_bwd_workspace_bytes(d))


def fwd(dims, **change):
    return call("ssm_delta_fwd", dims, FWD, **change)


def step(dims, **change):
    return call("ssm_delta_step", dims, STEP, **change)


def grads(**change):
    g = ssm.SsmDeltaGrads(at(20), at(21), at(22), at(23), at(24), None)
    for k, v in change.items():
        setattr(g, k, v)
    return g


def bwd(dims, into=None, **change):
    return call("ssm_delta_bwd", dims, BWD, (into or grads(),), **change)


def test_null_and_empty():
    assert fwd(None) == ssm.SSM_ERR_NULL
    for p in ("q", "k", "v", "g", "beta", "o"):
        assert fwd(ready(), **{p: None}) == ssm.SSM_ERR_NULL
    assert fwd(ready(), **{"-slots": at(30)}) == ssm.SSM_ERR_NULL           # slots without states
    for p in ("q", "k", "v", "g", "beta", "states", "o"):
        assert step(lin(tokens=2, nslots=2), **{p: None}) == ssm.SSM_ERR_NULL
    for p in ("q", "k", "v", "g", "beta", "do"):
        assert bwd(ready_b(), **{p: None}) == ssm.SSM_ERR_NULL
    for p in ("dq", "dk", "dv", "dg", "dbeta"):
        assert bwd(ready_b(), grads(**{p: None})) == ssm.SSM_ERR_NULL
    assert bwd(ready_b(), **{"-s0": at(30)}) == ssm.SSM_ERR_NULL            # s0 without ds0
    for field in ("tokens", "nseq", "nheads", "kheads", "dk", "dv"):
        for v in (0, -3):
            assert fwd(lin(**{field: v})) == ssm.SSM_ERR_EMPTY
            assert bwd(lin(**{field: v})) == ssm.SSM_ERR_EMPTY
            assert step(lin(**{field: v})) == ssm.SSM_ERR_EMPTY
            assert ssm.ssm_delta_fwd_workspace_bytes(lin(**{field: v})) == 0
            assert ssm.ssm_delta_bwd_workspace_bytes(lin(**{field: v})) == 0


@pytest.mark.parametrize("bad", [dict(kheads=3), dict(dk=257), dict(dv=257), dict(nseq=65536), dict(nheads=32768, kheads=1),
                                 dict(tokens=1 << 31), dict(head_decay=2), dict(reserved=1), dict(piece_len=-64),
                                 dict(piece_len=100), dict(piece_len=32), dict(q_stride=127), dict(k_stride=1), dict(v_stride=127),
                                 dict(o_stride=100), dict(q_stride=1 << 40), dict(o_stride=1 << 23), dict(nseq=3)])
def test_sizes(bad):
    assert fwd(ready(**bad)) == ssm.SSM_ERR_DIMS
    assert bwd(ready_b(**bad)) == ssm.SSM_ERR_DIMS
    if "nseq" not in bad or bad["nseq"] != 3:
        assert ssm.ssm_delta_fwd_workspace_bytes(lin(**bad)) == 0
        assert ssm.ssm_delta_bwd_workspace_bytes(lin(**bad)) == 0


def test_states_types_and_alignment():
    assert fwd(lin(io_dtype=7)) == ssm.SSM_ERR_DTYPE
    assert bwd(lin(io_dtype=7)) == ssm.SSM_ERR_DTYPE
    for n in (0, 1, -1):
        assert fwd(ready(nslots=n), **{"-s0": at(30)}) == ssm.SSM_ERR_DIMS   # fewer states than sequences
    assert step(lin(nslots=100)) == ssm.SSM_ERR_DIMS                         # tokens != nseq
    assert step(lin(tokens=2, nslots=1)) == ssm.SSM_ERR_DIMS
    for names, run, make in ((FWD, fwd, ready), (STEP, step, lambda **k: lin(tokens=2, nslots=2, **k)), (BWD, bwd, ready_b)):
        for i, p in enumerate(names):
            if p in ("q", "k", "v", "o", "g", "beta", "states", "do"):
                assert run(make(), **{p: at(i, 1)}) == ssm.SSM_ERR_ALIGN
                assert run(make(io_dtype=0), **{p: at(i, 2)}) == ssm.SSM_ERR_ALIGN
    for p in ("-cu", "-slots", "-s0", "-s_last"):
        assert fwd(ready(nslots=2), **{"-s0": at(30), p: at(31, 2)}) == ssm.SSM_ERR_ALIGN
    for p in ("dq", "dk", "dv"):
        assert bwd(ready_b(), grads(**{p: at(30, 1)})) == ssm.SSM_ERR_ALIGN
    for p in ("dg", "dbeta", "ds0"):
        assert bwd(ready_b(), grads(**{p: at(30, 2)})) == ssm.SSM_ERR_ALIGN


def test_workspace_and_overlaps():
    need = ssm.ssm_delta_fwd_workspace_bytes(lin())
    assert need > 0 and fwd(lin()) == ssm.SSM_ERR_WORKSPACE                  # always needed
    dense = ssm.ssm_delta_fwd_workspace_bytes(lin(tokens=96, nseq=1))
    d = lin(tokens=4096, nseq=1, nheads=2, kheads=2, dk=64, dv=64, piece_len=64)
    need = ssm.ssm_delta_fwd_workspace_bytes(d)
    assert need > dense
    assert fwd(with_workspace(d, need // 2)) == ssm.SSM_ERR_WORKSPACE
    d.workspace_bytes = need
    d.workspace = at(40, 128)
    assert fwd(d) == ssm.SSM_ERR_WORKSPACE
    for i in (0, 1, 2, 3, 4, 8):
        d.workspace = at(i)
        assert fwd(d) == ssm.SSM_ERR_ALIAS
    for i in (0, 1, 2, 3, 4):
        assert fwd(ready(), o=at(i)) == ssm.SSM_ERR_ALIAS
    row = 2 * 64 + 4 * 32
    assert fwd(ready(q_stride=row, o_stride=row), o=at(0, 2 * 2 * 64 - 2)) == ssm.SSM_ERR_ALIAS
    assert fwd(ready(nslots=2), **{"-s0": at(30), "-s_last": at(30, 4)}) == ssm.SSM_ERR_ALIAS
    assert fwd(ready(nslots=2), **{"-s0": at(30), "-s_last": at(8)}) == ssm.SSM_ERR_ALIAS
    for i in (0, 1, 2, 3, 4, 7):
        assert step(lin(tokens=2, nslots=2), states=at(i)) == ssm.SSM_ERR_ALIAS
    need = ssm.ssm_delta_bwd_workspace_bytes(lin())
    assert need > 0 and bwd(lin()) == ssm.SSM_ERR_WORKSPACE
    assert bwd(with_workspace(lin(), need // 2)) == ssm.SSM_ERR_WORKSPACE
    for name in ("dq", "dk", "dv", "dg", "dbeta", "ds0"):
        for i in (0, 1, 2, 3, 4, 7, 21 if name != "dk" else 20, 40):
            assert bwd(ready_b(), grads(**{name: at(i)})) == ssm.SSM_ERR_ALIAS, (name, i)
    d = ready_b()
    d.workspace = at(23)
    assert bwd(d) == ssm.SSM_ERR_ALIAS


@pytest.mark.parametrize("lens", [(4096, 1), (4096, 4), (100, 2), (64, 64), (131072, 1), (1, 1)])
def test_one_workspace_covers_packed_and_even_sequences(lens):
    """What the size functions ask for is enough with cu_seqlens and without: a call on it gets
    as far as the check of overlaps, one on less does not."""
    for piece in (0, 64, 1024):
        kw = dict(tokens=lens[0], nseq=lens[1], nheads=8, kheads=2, dk=128, dv=128, piece_len=piece)
        for cu in (None, at(30)):
            assert fwd(ready(**kw), o=at(0), **{"-cu": cu}) == ssm.SSM_ERR_ALIAS
            assert bwd(ready_b(**kw), grads(dq=at(0)), **{"-cu": cu}) == ssm.SSM_ERR_ALIAS
            d = ready(**kw)
            d.workspace_bytes = 0
            assert fwd(d, o=at(0), **{"-cu": cu}) == ssm.SSM_ERR_WORKSPACE


def layer(rows=10, dim=64, x_stride=0, y_stride=0, io=1, eps=1e-5, ws=None, bytes_=0):
    return ssm.SsmLayerNormDims(rows, dim, x_stride, y_stride, io, eps, ws, bytes_)


def test_layer_norm_refusals():
    assert call("ssm_layer_norm_fwd", None, LAYER) == ssm.SSM_ERR_NULL
    assert call("ssm_layer_norm_bwd", None, LAYER_B) == ssm.SSM_ERR_NULL
    for p in ("x", "w", "y"):
        assert call("ssm_layer_norm_fwd", layer(), LAYER, **{p: None}) == ssm.SSM_ERR_NULL
    for p in ("x", "w", "dy", "dx", "dw"):
        assert call("ssm_layer_norm_bwd", layer(), LAYER_B, **{p: None}) == ssm.SSM_ERR_NULL
    for bad in (dict(rows=0), dict(dim=0), dict(dim=-1)):
        assert call("ssm_layer_norm_fwd", layer(**bad), LAYER) == ssm.SSM_ERR_EMPTY
        assert ssm.ssm_layer_norm_bwd_workspace_bytes(layer(**bad)) == 0
    for bad in (dict(dim=16385), dict(x_stride=63), dict(y_stride=-5), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-40),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=1 << 41), dict(x_stride=1 << 40)):
        assert call("ssm_layer_norm_fwd", layer(**bad), LAYER) == ssm.SSM_ERR_DIMS
        assert call("ssm_layer_norm_bwd", layer(**bad), LAYER_B) == ssm.SSM_ERR_DIMS
        assert ssm.ssm_layer_norm_bwd_workspace_bytes(layer(**bad)) == 0
    assert call("ssm_layer_norm_fwd", layer(io=2), LAYER) == ssm.SSM_ERR_DTYPE
    for i, p in enumerate(LAYER):
        assert call("ssm_layer_norm_fwd", layer(), LAYER, **{p: at(i, 1)}) == ssm.SSM_ERR_ALIGN
    for i, p in enumerate(LAYER_B):
        assert call("ssm_layer_norm_bwd", layer(), LAYER_B, **{p: at(i, 1)}) == ssm.SSM_ERR_ALIGN
    assert call("ssm_layer_norm_bwd", layer(), LAYER_B) == ssm.SSM_ERR_WORKSPACE
    for bad in (dict(y=at(1)), dict(y=at(0, 16)), {"-b": at(3)}):
        assert call("ssm_layer_norm_fwd", layer(), LAYER, **bad) == ssm.SSM_ERR_ALIAS
    assert call("ssm_layer_norm_fwd", layer(y_stride=200), LAYER, y=at(0)) == ssm.SSM_ERR_ALIAS
    need = ssm.ssm_layer_norm_bwd_workspace_bytes(layer())
    assert need > 0
    for bad in (dict(dx=at(0)), dict(dx=at(2)), dict(dw=at(1)), dict(dw=at(3)), {"-db": at(4)}, {"-db": at(40)}):
        assert call("ssm_layer_norm_bwd", layer(ws=at(40), bytes_=need), LAYER_B, **bad) == ssm.SSM_ERR_ALIAS
    assert call("ssm_layer_norm_bwd", layer(ws=at(40), bytes_=need - 1), LAYER_B) == ssm.SSM_ERR_WORKSPACE


def test_binding_checks_its_arguments():
    import torch

    q, b = torch.zeros(8, 2, 16), torch.zeros(8, 2)
    for run in (lambda: ssm.delta_fwd(q, q, q, b, b), lambda: ssm.delta_step(q, q, q, b, b, torch.zeros(8, 2, 16, 16)),
                lambda: ssm.delta_bwd(q, q, q, b, b, do=q), lambda: ssm.layer_norm_fwd(q, torch.zeros(16)),
                lambda: ssm.layer_norm_bwd(q, torch.zeros(16), dy=q)):
        with pytest.raises(ValueError, match="device"):
            run()
    # the checks behind the device's, on the CPU
    dims = ssm.blocks._delta_dims(q, q, torch.zeros(8, 4, 24), torch.zeros(8, 4), torch.zeros(8, 4), 0.5, None)
    assert (dims.tokens, dims.nseq, dims.nheads, dims.kheads, dims.dk, dims.dv, dims.head_decay) == (8, 1, 4, 2, 16, 24, 0)
    d4 = ssm.blocks._delta_dims(q.view(2, 4, 2, 16), q.view(2, 4, 2, 16), q.view(2, 4, 2, 16), torch.zeros(2),
                                torch.zeros(2, 4, 2), 1.0, None)
    assert (d4.tokens, d4.nseq, d4.head_decay) == (8, 2, 1)
    for bad in (torch.zeros(8, 3), torch.zeros(2), torch.zeros(8, 1).expand(8, 2), torch.zeros(7, 2)):
        with pytest.raises(ValueError, match="beta"):
            ssm.blocks._delta_dims(q, q, q, b, bad, 1.0, None)
    with pytest.raises(TypeError, match="beta"):
        ssm.blocks._delta_dims(q, q, q, b, b.bfloat16(), 1.0, None)
    for bad in (torch.zeros(15), torch.zeros(2, 16)):
        with pytest.raises(ValueError, match="weight"):
            ssm.blocks._layer_dims(q, bad, None, 1e-5)
        with pytest.raises(ValueError, match="bias"):
            ssm.blocks._layer_dims(q, torch.zeros(16), bad, 1e-5)
    with pytest.raises(TypeError):
        ssm.blocks._layer_dims(q, torch.zeros(16).bfloat16(), None, 1e-5)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ssm.blocks._layer_dims(q.half(), torch.zeros(16), None, 1e-5)
    with pytest.raises(ValueError, match="rows"):
        ssm.blocks._layer_dims(torch.zeros(16), torch.zeros(16), None, 1e-5)


class Stream:
    cuda_stream, device_index = 0x1234, 1


@pytest.mark.parametrize("name,count", [("ssm_delta_fwd", 10), ("ssm_delta_step", 8), ("ssm_delta_bwd", 10), ("ssm_layer_norm_fwd", 4),
                                        ("ssm_layer_norm_bwd", 6)])
def test_stream_of_another_device(name, count, monkeypatch):
    calls = []
    monkeypatch.setitem(ssm.blocks._bound, name, lambda *a: calls.append(a) or 0)
    with pytest.raises(ValueError, match="stream"):
        ssm.blocks._call(name, (None,) * count, 0, Stream())
    assert not calls
