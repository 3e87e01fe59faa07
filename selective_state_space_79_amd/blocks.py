"""The operators of a block around a recurrent mixer, as bound from libssm.so: linear
attention with a decay for each head (``linattn_fwd``, ``linattn_step``, ``linattn_bwd``), the
gated delta rule (``delta_fwd``, ``delta_step``, ``delta_bwd``) and the norms before and after a
block (``gated_norm_fwd``, ``gated_norm_bwd``, ``add_norm_fwd``, ``add_norm_bwd``,
``layer_norm_fwd``, ``layer_norm_bwd``).

Argument marshalling only, like the rest of the package; include/ssm.h states what each call
computes.  The ``ssm_*`` functions carry the C names, take the tensors of the call (or None)
and a dims struct, and return the status; the others check their arguments, allocate outputs
and workspaces with torch on the stream of the call and raise SsmError on a refused call.
"""
from __future__ import annotations

import contextlib
import ctypes

__all__ = ["SSM_LINATTN_MAX_DIM", "SSM_NORM_MAX_DIM", "SsmLinattnDims", "SsmLinattnGrads", "SsmGatedNormDims",
           "SsmAddNormDims", "make_linattn_dims", "linattn_fwd", "linattn_step", "linattn_bwd", "gated_norm_fwd",
           "gated_norm_bwd", "add_norm_fwd", "add_norm_bwd", "ssm_linattn_fwd", "ssm_linattn_step", "ssm_linattn_bwd",
           "ssm_linattn_fwd_workspace_bytes", "ssm_linattn_bwd_workspace_bytes", "ssm_gated_norm_fwd",
           "ssm_gated_norm_bwd", "ssm_gated_norm_bwd_workspace_bytes", "ssm_add_norm_fwd", "ssm_add_norm_bwd",
           "ssm_add_norm_bwd_workspace_bytes", "SsmDeltaGrads", "SsmLayerNormDims", "delta_fwd", "delta_step",
           "delta_bwd", "layer_norm_fwd", "layer_norm_bwd", "ssm_delta_fwd", "ssm_delta_step", "ssm_delta_bwd",
           "ssm_delta_fwd_workspace_bytes", "ssm_delta_bwd_workspace_bytes", "ssm_layer_norm_fwd",
           "ssm_layer_norm_bwd", "ssm_layer_norm_bwd_workspace_bytes"]

_vp = ctypes.c_void_p
_ref = ctypes.byref
_i64, _i32, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_float

SSM_LINATTN_MAX_DIM = 256
SSM_NORM_MAX_DIM = 16384


class SsmLinattnDims(ctypes.Structure):
    """Mirror of ``ssm_linattn_dims`` in include/ssm.h."""
    _fields_ = [("tokens", _i64), ("nseq", _i64), ("nheads", _i64), ("kheads", _i64), ("dk", _i64), ("dv", _i64),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("o_stride", _i64), ("nslots", _i64),
                ("piece_len", _i64), ("io_dtype", _i32), ("head_decay", _i32), ("scale", _f32), ("reserved", _i32),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class SsmLinattnGrads(ctypes.Structure):
    """Mirror of ``ssm_linattn_grads`` in include/ssm.h (device pointers; None = NULL)."""
    _fields_ = [(name, _vp) for name in ("dq", "dk", "dv", "dg", "ds0")]


class SsmGatedNormDims(ctypes.Structure):
    """Mirror of ``ssm_gated_norm_dims`` in include/ssm.h."""
    _fields_ = [("rows", _i64), ("ngroups", _i64), ("group", _i64), ("x_stride", _i64), ("z_stride", _i64),
                ("y_stride", _i64), ("io_dtype", _i32), ("gate_first", _i32), ("shared_weight", _i32), ("eps", _f32),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class SsmAddNormDims(ctypes.Structure):
    """Mirror of ``ssm_add_norm_dims`` in include/ssm.h."""
    _fields_ = [("rows", _i64), ("dim", _i64), ("x_stride", _i64), ("res_stride", _i64), ("r_stride", _i64),
                ("y_stride", _i64), ("io_dtype", _i32), ("res_dtype", _i32), ("eps", _f32), ("reserved", _i32),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class SsmDeltaGrads(ctypes.Structure):
    """Mirror of ``ssm_delta_grads`` in include/ssm.h (device pointers; None = NULL)."""
    _fields_ = [(name, _vp) for name in ("dq", "dk", "dv", "dg", "dbeta", "ds0")]


class SsmLayerNormDims(ctypes.Structure):
    """Mirror of ``ssm_layer_norm_dims`` in include/ssm.h."""
    _fields_ = [("rows", _i64), ("dim", _i64), ("x_stride", _i64), ("y_stride", _i64), ("io_dtype", _i32), ("eps", _f32),
                ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


# C name -> (pointers before the struct arguments, struct types); a stream follows
_CALLS = {
    "ssm_linattn_fwd": (9, (SsmLinattnDims,)),
    "ssm_linattn_step": (7, (SsmLinattnDims,)),
    "ssm_linattn_bwd": (8, (SsmLinattnGrads, SsmLinattnDims)),
    "ssm_gated_norm_fwd": (4, (SsmGatedNormDims,)),
    "ssm_gated_norm_bwd": (7, (SsmGatedNormDims,)),
    "ssm_add_norm_fwd": (7, (SsmAddNormDims,)),
    "ssm_add_norm_bwd": (12, (SsmAddNormDims,)),
    "ssm_delta_fwd": (10, (SsmLinattnDims,)),
    "ssm_delta_step": (8, (SsmLinattnDims,)),
    "ssm_delta_bwd": (9, (SsmDeltaGrads, SsmLinattnDims)),
    "ssm_layer_norm_fwd": (4, (SsmLayerNormDims,)),
    "ssm_layer_norm_bwd": (6, (SsmLayerNormDims,)),
}
_SIZES = {
    "ssm_linattn_fwd_workspace_bytes": SsmLinattnDims,
    "ssm_linattn_bwd_workspace_bytes": SsmLinattnDims,
    "ssm_gated_norm_bwd_workspace_bytes": SsmGatedNormDims,
    "ssm_add_norm_bwd_workspace_bytes": SsmAddNormDims,
    "ssm_delta_fwd_workspace_bytes": SsmLinattnDims,
    "ssm_delta_bwd_workspace_bytes": SsmLinattnDims,
    "ssm_layer_norm_bwd_workspace_bytes": SsmLayerNormDims,
}
EXPORTED = tuple(_CALLS) + tuple(_SIZES)


def declare(lib):
    """Argument types of this module's entry points (called once by load_library)."""
    for name, (n, structs) in _CALLS.items():
        f = getattr(lib, name)
        f.argtypes = [_vp] * n + [ctypes.POINTER(s) for s in structs] + [_vp]
        f.restype = ctypes.c_int
    for name, s in _SIZES.items():
        f = getattr(lib, name)
        f.argtypes = [ctypes.POINTER(s)]
        f.restype = ctypes.c_size_t


_bound = {}     # C name -> function of the loaded library


def _package():
    import selective_state_space_79_amd as ssm

    return ssm


def _fn(name):
    f = _bound.get(name)
    if f is None:
        f = _bound[name] = getattr(_package().load_library(), name)
    return f


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, args, device, stream):
    """Calls a C entry point; args: pointers and struct references, before the stream."""
    import torch

    f = _fn(name)
    index = device if device >= 0 else torch.cuda.current_device()
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        _need(stream.device_index == index, f"stream must be one of cuda:{index}, the tensors' device")
        raw = stream.cuda_stream
    # a launch goes to the current device, so that has to be the tensors'
    if index == torch._C._cuda_getDevice():
        return f(*args, raw)
    with torch.cuda.device(index):
        return f(*args, raw)


def ssm_linattn_fwd(q, k, v, g, cu_seqlens, slots, s0, o, s_last, dims, stream=None) -> int:
    """C entry point of the forward; returns the status."""
    return _call("ssm_linattn_fwd", (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(cu_seqlens),
                                     _ptr(slots), _ptr(s0), o.data_ptr(), _ptr(s_last), _ref(dims)),
                 q.get_device(), stream)


def ssm_linattn_step(q, k, v, g, slots, states, o, dims, stream=None) -> int:
    """C entry point of the single-token step; returns the status."""
    return _call("ssm_linattn_step", (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(slots),
                                      states.data_ptr(), o.data_ptr(), _ref(dims)), q.get_device(), stream)


def ssm_linattn_bwd(q, k, v, g, cu_seqlens, s0, do, ds_last, grads, dims, stream=None) -> int:
    """C entry point of the gradients; returns the status."""
    return _call("ssm_linattn_bwd", (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(cu_seqlens),
                                     _ptr(s0), do.data_ptr(), _ptr(ds_last), _ref(grads), _ref(dims)),
                 q.get_device(), stream)


def ssm_gated_norm_fwd(x, z, w, y, dims, stream=None) -> int:
    """C entry point of the gated norm; returns the status."""
    return _call("ssm_gated_norm_fwd", (x.data_ptr(), _ptr(z), w.data_ptr(), y.data_ptr(), _ref(dims)),
                 x.get_device(), stream)


def ssm_gated_norm_bwd(x, z, w, dy, dx, dz, dw, dims, stream=None) -> int:
    """C entry point of the gated norm's gradients; returns the status."""
    return _call("ssm_gated_norm_bwd", (x.data_ptr(), _ptr(z), w.data_ptr(), dy.data_ptr(), dx.data_ptr(), _ptr(dz),
                                        dw.data_ptr(), _ref(dims)), x.get_device(), stream)


def ssm_add_norm_fwd(x, res, scale, post, w, r, y, dims, stream=None) -> int:
    """C entry point of the residual addition with its norms; returns the status."""
    return _call("ssm_add_norm_fwd", (x.data_ptr(), _ptr(res), _ptr(scale), _ptr(post), w.data_ptr(), r.data_ptr(),
                                      y.data_ptr(), _ref(dims)), x.get_device(), stream)


def ssm_add_norm_bwd(x, r, scale, post, w, dy, dr, dx, dres, dw, dscale, dpost, dims, stream=None) -> int:
    """C entry point of the residual addition's gradients; returns the status."""
    return _call("ssm_add_norm_bwd", (_ptr(x), r.data_ptr(), _ptr(scale), _ptr(post), w.data_ptr(), dy.data_ptr(),
                                      _ptr(dr), dx.data_ptr(), _ptr(dres), dw.data_ptr(), _ptr(dscale), _ptr(dpost),
                                      _ref(dims)), r.get_device(), stream)


def ssm_linattn_fwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_linattn_fwd_workspace_bytes")(_ref(dims)))


def ssm_linattn_bwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_linattn_bwd_workspace_bytes")(_ref(dims)))


def ssm_gated_norm_bwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_gated_norm_bwd_workspace_bytes")(_ref(dims)))


def ssm_add_norm_bwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_add_norm_bwd_workspace_bytes")(_ref(dims)))


def ssm_delta_fwd(q, k, v, g, beta, cu_seqlens, slots, s0, o, s_last, dims, stream=None) -> int:
    """C entry point of the delta rule's forward; returns the status."""
    return _call("ssm_delta_fwd", (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                   _ptr(cu_seqlens), _ptr(slots), _ptr(s0), o.data_ptr(), _ptr(s_last), _ref(dims)),
                 q.get_device(), stream)


def ssm_delta_step(q, k, v, g, beta, slots, states, o, dims, stream=None) -> int:
    """C entry point of the delta rule's single-token step; returns the status."""
    return _call("ssm_delta_step", (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(slots),
                                    states.data_ptr(), o.data_ptr(), _ref(dims)), q.get_device(), stream)


def ssm_delta_bwd(q, k, v, g, beta, cu_seqlens, s0, do, ds_last, grads, dims, stream=None) -> int:
    """C entry point of the delta rule's gradients; returns the status."""
    return _call("ssm_delta_bwd", (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                   _ptr(cu_seqlens), _ptr(s0), do.data_ptr(), _ptr(ds_last), _ref(grads), _ref(dims)),
                 q.get_device(), stream)


def ssm_layer_norm_fwd(x, w, b, y, dims, stream=None) -> int:
    """C entry point of the layer norm; returns the status."""
    return _call("ssm_layer_norm_fwd", (x.data_ptr(), w.data_ptr(), _ptr(b), y.data_ptr(), _ref(dims)), x.get_device(),
                 stream)


def ssm_layer_norm_bwd(x, w, dy, dx, dw, db, dims, stream=None) -> int:
    """C entry point of the layer norm's gradients; returns the status."""
    return _call("ssm_layer_norm_bwd", (x.data_ptr(), w.data_ptr(), dy.data_ptr(), dx.data_ptr(), dw.data_ptr(), _ptr(db),
                                        _ref(dims)), x.get_device(), stream)


def ssm_delta_fwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_delta_fwd_workspace_bytes")(_ref(dims)))


def ssm_delta_bwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_delta_bwd_workspace_bytes")(_ref(dims)))


def ssm_layer_norm_bwd_workspace_bytes(dims) -> int:
    return int(_fn("ssm_layer_norm_bwd_workspace_bytes")(_ref(dims)))


# ------------------------------------------------------------------ checks
def _io(name, t):
    import torch

    if t.dtype is torch.bfloat16:
        return 1
    if t.dtype is torch.float32:
        return 0
    raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}")


def _need(cond, text):
    if not cond:
        raise ValueError(text)


def _device(ref, *tensors):
    """All on ref's device, which is a GPU.  The checks of this module run before every call
    of a few microseconds: they touch each tensor once."""
    d = ref.get_device()
    if d < 0:
        raise ValueError("device tensors are needed")
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError(f"all tensors must be on {ref.device}")


def _dense(name, t, dtype, *shapes):
    """A contiguous tensor of one of these shapes."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape not in shapes:
        raise ValueError(f"{name} must be {' or '.join(map(str, shapes))}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _step(name, t, sh):
    """Elements between the tokens of a (T, heads, width) or (batch, L, heads, width) tensor
    whose heads are contiguous within a token (0: packed)."""
    if t.is_contiguous():
        return 0
    st = t.stride()
    heads, width = sh[-2], sh[-1]
    if not ((width == 1 or st[-1] == 1) and (heads == 1 or st[-2] == width)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if len(sh) == 4 and sh[0] > 1 and sh[1] > 1 and st[0] != sh[1] * st[1]:
        raise ValueError(f"{name}: batch rows must follow one another")
    tokens = next(((n, s) for n, s in zip(sh[-3::-1], st[-3::-1]) if n > 1), None)
    return 0 if tokens is None else _apart(name, tokens[1], heads * width)


def _apart(name, step, width):
    """A step between rows that is one (0 would be taken for packed rows)."""
    if step < width:
        raise ValueError(f"{name}: rows must not overlap (an expanded tensor has to be copied first)")
    return step


_HERE = contextlib.nullcontext()


def _on(stream):
    """Allocations for a call on another stream belong to that stream."""
    import torch

    return _HERE if stream is None else torch.cuda.stream(stream)


def _workspace(need, given, device):
    """The caller's workspace, or a new one if that is too small, and its bytes.  A view whose
    elements are strided or expanded is not memory of its own size."""
    import torch

    if need == 0:
        return None, 0
    if given is not None:
        _need(given.device == device, f"workspace must be on {device}")
        _need(given.is_contiguous(), "workspace must be contiguous")
    if given is None or given.numel() * given.element_size() < need:
        given = torch.empty(need, dtype=torch.uint8, device=device)
    return given, given.numel() * given.element_size()


def _ok(st, where):
    if st != 0:
        raise _package().SsmError(st, where)


# ------------------------------------------------------------------ linear attention
def make_linattn_dims(tokens, nseq, nheads, kheads, dk, dv, *, io_dtype=1, scale=1.0, head_decay=0, q_stride=0,
                      k_stride=0, v_stride=0, o_stride=0, nslots=0, piece_len=0, workspace=0, workspace_bytes=0,
                      reserved=0) -> SsmLinattnDims:
    return SsmLinattnDims(tokens, nseq, nheads, kheads, dk, dv, q_stride, k_stride, v_stride, o_stride, nslots,
                          piece_len, io_dtype, head_decay, scale, reserved, workspace or None, workspace_bytes)


def _linattn_dims(q, k, v, g, scale, nseq):
    import torch

    sq, sk, sv = q.shape, k.shape, v.shape
    if len(sq) not in (3, 4):
        raise ValueError("q, k and v must all be (tokens, heads, d) or all (batch, L, heads, d)")
    if sq != sk or sq[:-2] != sv[:-2] or len(sv) != len(sq):
        raise ValueError("q and k must have one shape, and v their tokens")
    dt = q.dtype
    if k.dtype is not dt or v.dtype is not dt:
        raise TypeError("q, k and v must have one dtype")
    heads = sv[-2]
    per_head = g.dim() == 1
    _dense("g", g, torch.float32, (heads,) if per_head else sv[:-1])
    n = sq[0]
    if len(sq) == 4:
        nseq, n = n, n * sq[1]
    return SsmLinattnDims(n, 1 if nseq is None else nseq, heads, sq[-2], sq[-1], sv[-1], _step("q", q, sq),
                          _step("k", k, sk), _step("v", v, sv), 0, 0, 0, _io("q", q), per_head, scale, 0, None, 0)


def _rows_out(out, like, dims):
    """The given output, or a new packed one, with its stride in dims."""
    import torch

    if out is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if out.dtype is not like.dtype or out.shape != like.shape:
        raise ValueError("out must have the shape and dtype of v")
    dims.o_stride = _step("out", out, out.shape)
    return out


def linattn_fwd(q, k, v, g, *, scale=1.0, cu_seqlens=None, s0=None, s_last=None, slots=None, return_state=False,
                out=None, workspace=None, piece_len=0, stream=None):
    """Linear attention with a decay for each head: S_t = e^{g_t} S_{t-1} + k_t v_t^T,
    o_t = scale S_t^T q_t.

    q, k: (tokens, kheads, dk) or (batch, L, kheads, dk); v: (.., heads, dv); a token's heads
    contiguous, any step from token to token.  g: float32 log decays (tokens, heads) (or
    (batch, L, heads)), or (heads,) for one decay per head.  cu_seqlens: int32 (nseq + 1),
    the starts of packed sequences (3-d tensors; without it they are one sequence).
    s0, s_last: float32 (nslots, heads, dk, dv) starting and final states; slots int32
    (nseq,) names each sequence's (default: in order); s_last may be s0, updated in place.
    With return_state and no s_last a new one is returned: (o, s_last).  Rows of no sequence,
    and of sequences whose slot is out of range or named before, are not written.
    """
    import torch

    _device(q, k, v, g, cu_seqlens, s0, s_last, slots, out, workspace)
    nseq = _packed(q, cu_seqlens)
    dims = _linattn_dims(q, k, v, g, scale, nseq)
    dims.piece_len = piece_len
    with _on(stream):
        if return_state or s0 is not None or s_last is not None:
            s_last = _states(dims, q, s0, s_last, slots, return_state)
        if slots is not None:
            _dense("slots", slots, torch.int32, (dims.nseq,))
        o = _rows_out(out, v, dims)
        need = _fn("ssm_linattn_fwd_workspace_bytes")(_ref(dims))
        if need:
            workspace, dims.workspace_bytes = _workspace(need, workspace, q.device)
            dims.workspace = workspace.data_ptr()
        st = ssm_linattn_fwd(q, k, v, g, cu_seqlens, slots, s0, o, s_last, dims, stream)
    if st:
        raise _package().SsmError(st, "ssm_linattn_fwd")
    return (o, s_last) if return_state else o


def _packed(q, cu_seqlens):
    import torch

    if cu_seqlens is None:
        return None
    _need(q.dim() == 3, "cu_seqlens needs packed (tokens, heads, d) tensors")
    n = cu_seqlens.numel()
    _dense("cu_seqlens", cu_seqlens, torch.int32, (n,))
    return n - 1


def _states(dims, q, s0, s_last, slots, make):
    """Checks the states of a forward call, and makes the final ones when asked for."""
    import torch

    state = (dims.nheads, dims.dk, dims.dv)
    if make and s_last is None:
        n = dims.nseq if slots is None else (s0.shape[0] if s0 is not None else None)
        _need(n is not None, "slots without states: give s0 or s_last")
        # states that no sequence names keep what they were
        s_last = torch.empty((n,) + state, dtype=torch.float32, device=q.device) if slots is None else s0.clone()
    for name, t in (("s0", s0), ("s_last", s_last)):
        if t is not None:
            dims.nslots = t.shape[0]
            _dense(name, t, torch.float32, (dims.nslots,) + state)
    if s0 is not None and s_last is not None:
        _need(s0.shape == s_last.shape, "s0 and s_last must have one shape")
    return s_last


def linattn_step(q, k, v, g, states, *, slots=None, scale=1.0, out=None, stream=None):
    """One token of each sequence: q, k (batch, kheads, dk), v (batch, heads, dv), g
    (batch, heads) or (heads,); states float32 (nslots, heads, dk, dv), updated in place;
    slots int32 (batch,) names each sequence's state (default: in order).  Rows whose slot is
    out of range or named before are skipped.  Returns o."""
    import torch

    _device(q, k, v, g, states, slots, out)
    sq = q.shape
    if len(sq) != 3:
        raise ValueError("q must be (batch, heads, dk)")
    dims = _linattn_dims(q, k, v, g, scale, sq[0])
    ss = states.shape
    dims.nslots = ss[0]
    _dense("states", states, torch.float32, (ss[0], v.shape[1], sq[2], v.shape[2]))
    if slots is not None:
        _dense("slots", slots, torch.int32, (sq[0],))
    with _on(stream):
        o = _rows_out(out, v, dims)
        st = ssm_linattn_step(q, k, v, g, slots, states, o, dims, stream)
    if st:
        raise _package().SsmError(st, "ssm_linattn_step")
    return o


def linattn_bwd(q, k, v, g, *, do, scale=1.0, cu_seqlens=None, s0=None, ds_last=None, workspace=None, piece_len=0,
                stream=None) -> dict:
    """Gradients of sum(do * o) + sum(ds_last * s_last) of linattn_fwd with the same inputs
    (states in the order of the sequences).  Returns a dict: dq, dk, dv (q's dtype), dg
    (float32, g's shape) and, with s0, ds0 (float32).  Rows of no sequence are zero."""
    import torch

    _device(q, k, v, g, do, cu_seqlens, s0, ds_last, workspace)
    nseq = _packed(q, cu_seqlens)
    dims = _linattn_dims(q, k, v, g, scale, nseq)
    dims.piece_len = piece_len
    if do.dtype is not v.dtype or do.shape != v.shape:
        raise ValueError("do must have the shape and dtype of v")
    dims.o_stride = _step("do", do, do.shape)
    state = (dims.nseq, dims.nheads, dims.dk, dims.dv)
    for name, t in (("s0", s0), ("ds_last", ds_last)):
        if t is not None:
            _dense(name, t, torch.float32, state)
    dims.nslots = dims.nseq
    dev = q.device
    with _on(stream):
        res = {"dq": torch.empty(q.shape, dtype=q.dtype, device=dev), "dk": torch.empty(k.shape, dtype=q.dtype, device=dev),
               "dv": torch.empty(v.shape, dtype=q.dtype, device=dev), "dg": torch.empty(g.shape, dtype=g.dtype, device=dev)}
        if s0 is not None:
            res["ds0"] = torch.empty(state, dtype=s0.dtype, device=dev)
        need = _fn("ssm_linattn_bwd_workspace_bytes")(_ref(dims))
        if need:
            workspace, dims.workspace_bytes = _workspace(need, workspace, dev)
            dims.workspace = workspace.data_ptr()
        grads = SsmLinattnGrads(*[_ptr(res.get(n)) for n, _ in SsmLinattnGrads._fields_])
        st = ssm_linattn_bwd(q, k, v, g, cu_seqlens, s0, do, ds_last, grads, dims, stream)
    _ok(st, "ssm_linattn_bwd")
    return res


# ------------------------------------------------------------------ the gated delta rule
def _delta_dims(q, k, v, g, beta, scale, nseq):
    import torch

    dims = _linattn_dims(q, k, v, g, scale, nseq)
    _dense("beta", beta, torch.float32, v.shape[:-1])
    return dims


def delta_fwd(q, k, v, g, beta, *, scale=1.0, cu_seqlens=None, s0=None, s_last=None, slots=None, return_state=False,
              out=None, workspace=None, piece_len=0, stream=None):
    """The gated delta rule: S' = e^{g_t} S_{t-1}, S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,
    o_t = scale S_t^T q_t.

    beta: float32 (tokens, heads) (or (batch, L, heads)); the other arguments, and what is
    returned, are those of linattn_fwd.  Keys are taken as they are: states stay bounded where
    0 <= beta |k|^2 <= 2.  The library cuts sequences by their mean length: for one long sequence
    packed with many short ones give piece_len (1024 to 4096, here and in delta_bwd).
    """
    import torch

    _device(q, k, v, g, beta, cu_seqlens, s0, s_last, slots, out, workspace)
    nseq = _packed(q, cu_seqlens)
    dims = _delta_dims(q, k, v, g, beta, scale, nseq)
    dims.piece_len = piece_len
    with _on(stream):
        if return_state or s0 is not None or s_last is not None:
            s_last = _states(dims, q, s0, s_last, slots, return_state)
        if slots is not None:
            _dense("slots", slots, torch.int32, (dims.nseq,))
        o = _rows_out(out, v, dims)
        need = _fn("ssm_delta_fwd_workspace_bytes")(_ref(dims))
        workspace, dims.workspace_bytes = _workspace(need, workspace, q.device)
        dims.workspace = _ptr(workspace)
        st = ssm_delta_fwd(q, k, v, g, beta, cu_seqlens, slots, s0, o, s_last, dims, stream)
    _ok(st, "ssm_delta_fwd")
    return (o, s_last) if return_state else o


def delta_step(q, k, v, g, beta, states, *, slots=None, scale=1.0, out=None, stream=None):
    """One token of each sequence: q, k (batch, kheads, dk), v (batch, heads, dv), g
    (batch, heads) or (heads,), beta (batch, heads); states float32 (nslots, heads, dk, dv),
    updated in place; slots int32 (batch,) names each sequence's state (default: in order).
    Rows whose slot is out of range or named before are skipped.  Returns o."""
    import torch

    _device(q, k, v, g, beta, states, slots, out)
    sq = q.shape
    if len(sq) != 3:
        raise ValueError("q must be (batch, heads, dk)")
    dims = _delta_dims(q, k, v, g, beta, scale, sq[0])
    ss = states.shape
    dims.nslots = ss[0]
    _dense("states", states, torch.float32, (ss[0], v.shape[1], sq[2], v.shape[2]))
    if slots is not None:
        _dense("slots", slots, torch.int32, (sq[0],))
    with _on(stream):
        o = _rows_out(out, v, dims)
        st = ssm_delta_step(q, k, v, g, beta, slots, states, o, dims, stream)
    _ok(st, "ssm_delta_step")
    return o


def delta_bwd(q, k, v, g, beta, *, do, scale=1.0, cu_seqlens=None, s0=None, ds_last=None, workspace=None, piece_len=0,
              stream=None) -> dict:
    """Gradients of sum(do * o) + sum(ds_last * s_last) of delta_fwd with the same inputs
    (states in the order of the sequences).  Returns a dict: dq, dk, dv (q's dtype), dg
    (float32, g's shape), dbeta (float32) and, with s0, ds0 (float32).  Rows of no sequence are
    zero."""
    import torch

    _device(q, k, v, g, beta, do, cu_seqlens, s0, ds_last, workspace)
    nseq = _packed(q, cu_seqlens)
    dims = _delta_dims(q, k, v, g, beta, scale, nseq)
    dims.piece_len = piece_len
    if do.dtype is not v.dtype or do.shape != v.shape:
        raise ValueError("do must have the shape and dtype of v")
    dims.o_stride = _step("do", do, do.shape)
    state = (dims.nseq, dims.nheads, dims.dk, dims.dv)
    for name, t in (("s0", s0), ("ds_last", ds_last)):
        if t is not None:
            _dense(name, t, torch.float32, state)
    dims.nslots = dims.nseq
    dev = q.device
    with _on(stream):
        res = {"dq": torch.empty(q.shape, dtype=q.dtype, device=dev), "dk": torch.empty(k.shape, dtype=q.dtype, device=dev),
               "dv": torch.empty(v.shape, dtype=q.dtype, device=dev), "dg": torch.empty(g.shape, dtype=g.dtype, device=dev),
               "dbeta": torch.empty(beta.shape, dtype=beta.dtype, device=dev)}
        if s0 is not None:
            res["ds0"] = torch.empty(state, dtype=s0.dtype, device=dev)
        need = _fn("ssm_delta_bwd_workspace_bytes")(_ref(dims))
        workspace, dims.workspace_bytes = _workspace(need, workspace, dev)
        dims.workspace = _ptr(workspace)
        grads = SsmDeltaGrads(*[_ptr(res.get(n)) for n, _ in SsmDeltaGrads._fields_])
        st = ssm_delta_bwd(q, k, v, g, beta, cu_seqlens, s0, do, ds_last, grads, dims, stream)
    _ok(st, "ssm_delta_bwd")
    return res


# ------------------------------------------------------------------ norms
def _matrix(name, t, sh):
    """Elements between the rows of a tensor whose leading dimensions collapse (0: packed)."""
    if len(sh) < 2:
        raise ValueError(f"{name} must have rows")
    if t.is_contiguous():
        return 0
    st = t.stride()
    if sh[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    rows, step = 1, None
    for n, s in zip(reversed(sh[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if step is not None and s != step * rows:
            raise ValueError(f"{name}: rows must be evenly spaced")
        if step is None:
            step = s
        rows *= n
    return 0 if step is None else _apart(name, step, sh[-1])


def _rows(t, sh):
    return sh[0] if len(sh) == 2 else t.numel() // max(1, sh[-1])


def _gated_dims(x, z, weight, group_size, gate_first, eps):
    import torch

    sh = x.shape
    sx, dim = _matrix("x", x, sh), sh[-1]
    group = dim if group_size is None else int(group_size)
    _need(group >= 1 and dim % group == 0, "group_size must divide x's last dimension")
    sz = 0
    if z is not None:
        if z.dtype is not x.dtype or z.shape != sh:
            raise ValueError("z must have the shape and dtype of x")
        sz = _matrix("z", z, sh)
    _dense("weight", weight, torch.float32, (dim,), (group,))
    shared = weight.numel() == group and group != dim
    return SsmGatedNormDims(_rows(x, sh), dim // group, group, sx, sz, 0, _io("x", x), bool(gate_first), shared, eps,
                            None, 0)


def gated_norm_fwd(x, z, weight, *, group_size=None, gate_first=True, eps=1e-5, out=None, stream=None):
    """RMS norm over groups of x's last dimension with a SiLU gate: norm(x SiLU(z)) weight
    with gate_first, else norm(x) weight SiLU(z); z may be None.  weight: float32 (dim,), or
    (group_size,) for every group; eps: 2^-126 or more.  out may be x or z.  Returns y, x's shape and dtype."""
    import torch

    _device(x, z, weight, out)
    dims = _gated_dims(x, z, weight, group_size, gate_first, eps)
    with _on(stream):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            if out.dtype is not x.dtype or out.shape != x.shape:
                raise ValueError("out must have the shape and dtype of x")
            dims.y_stride = _matrix("out", out, out.shape)
        _ok(ssm_gated_norm_fwd(x, z, weight, out, dims, stream), "ssm_gated_norm_fwd")
    return out


def gated_norm_bwd(x, z, weight, *, dy, group_size=None, gate_first=True, eps=1e-5, workspace=None,
                   stream=None) -> dict:
    """Gradients of sum(dy * y) of gated_norm_fwd: dx, dz (x's dtype; dz only with z) and
    dweight (float32)."""
    import torch

    _device(x, z, weight, dy, workspace)
    dims = _gated_dims(x, z, weight, group_size, gate_first, eps)
    _dense("dy", dy, x.dtype, x.shape)
    with _on(stream):
        res = {"dx": torch.empty(x.shape, dtype=x.dtype, device=x.device)}
        if z is not None:
            res["dz"] = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        res["dweight"] = torch.empty_like(weight)
        need = ssm_gated_norm_bwd_workspace_bytes(dims)
        workspace, dims.workspace_bytes = _workspace(need, workspace, x.device)
        dims.workspace = _ptr(workspace)
        _ok(ssm_gated_norm_bwd(x, z, weight, dy, res["dx"], res.get("dz"), res["dweight"], dims, stream),
            "ssm_gated_norm_bwd")
    return res


def _add_dims(x, res, weight, scale, post_weight, eps):
    import torch

    sh = x.shape
    sx, dim = _matrix("x", x, sh), sh[-1]
    _dense("weight", weight, torch.float32, (dim,))
    if scale is not None:
        _dense("scale", scale, torch.float32, (dim,))
    if post_weight is not None:
        _dense("post_weight", post_weight, torch.float32, (dim,))
    io = _io("x", x)
    sres, rt = 0, io
    if res is not None:
        if res.shape != sh:
            raise ValueError("the residual must have x's shape")
        rt = _io("residual", res)
        sres = _matrix("residual", res, sh)
    return SsmAddNormDims(_rows(x, sh), dim, sx, sres, 0, 0, io, rt, eps, 0, None, 0)


def add_norm_fwd(x, residual, weight, *, scale=None, post_weight=None, eps=1e-5, residual_out=None, out=None,
                 stream=None):
    """r = residual + scale * (x, or with post_weight its RMS norm); y = the RMS norm of r
    with weight.  residual: x's dtype or float32, or None (zeros; residual_out then tells
    r's dtype, else x's); scale, post_weight, weight: float32 (dim,); eps: 2^-126 or more.
    residual_out may be residual.  Returns (y, r)."""
    import torch

    _device(x, residual, weight, scale, post_weight, residual_out, out)
    dims = _add_dims(x, residual, weight, scale, post_weight, eps)
    with _on(stream):
        if residual_out is None:
            residual_out = torch.empty(x.shape, dtype=x.dtype if residual is None else residual.dtype, device=x.device)
        else:
            if residual_out.shape != x.shape or (residual is not None and residual_out.dtype is not residual.dtype):
                raise ValueError("residual_out must have x's shape and the residual's dtype")
            dims.res_dtype = _io("residual_out", residual_out)
            dims.r_stride = _matrix("residual_out", residual_out, residual_out.shape)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            if out.dtype is not x.dtype or out.shape != x.shape:
                raise ValueError("out must have the shape and dtype of x")
            dims.y_stride = _matrix("out", out, out.shape)
        _ok(ssm_add_norm_fwd(x, residual, scale, post_weight, weight, residual_out, out, dims, stream),
            "ssm_add_norm_fwd")
    return out, residual_out


def add_norm_bwd(x, r, weight, *, dy, dr=None, scale=None, post_weight=None, eps=1e-5, workspace=None,
                 stream=None) -> dict:
    """Gradients of sum(dy * y) + sum(dr * r) of add_norm_fwd, from x and the r it returned:
    dx (x's dtype), dresidual (r's dtype), dweight and, with scale and post_weight, dscale
    and dpost_weight (float32)."""
    import torch

    _device(x, r, weight, dy, dr, scale, post_weight, workspace)
    dims = _add_dims(x, r, weight, scale, post_weight, eps)
    dims.r_stride, dims.res_stride = dims.res_stride, 0
    _dense("dy", dy, x.dtype, x.shape)
    if dr is not None:
        _dense("dr", dr, r.dtype, r.shape)
    with _on(stream):
        res = {"dx": torch.empty(x.shape, dtype=x.dtype, device=x.device),
               "dresidual": torch.empty(x.shape, dtype=r.dtype, device=x.device), "dweight": torch.empty_like(weight)}
        if scale is not None:
            res["dscale"] = torch.empty_like(scale)
        if post_weight is not None:
            res["dpost_weight"] = torch.empty_like(post_weight)
        need = ssm_add_norm_bwd_workspace_bytes(dims)
        workspace, dims.workspace_bytes = _workspace(need, workspace, x.device)
        dims.workspace = _ptr(workspace)
        _ok(ssm_add_norm_bwd(x, r, scale, post_weight, weight, dy, dr, res["dx"], res["dresidual"], res["dweight"],
                             res.get("dscale"), res.get("dpost_weight"), dims, stream), "ssm_add_norm_bwd")
    return res


def _layer_dims(x, weight, bias, eps):
    import torch

    sh = x.shape
    sx, dim = _matrix("x", x, sh), sh[-1]
    _dense("weight", weight, torch.float32, (dim,))
    if bias is not None:
        _dense("bias", bias, torch.float32, (dim,))
    return SsmLayerNormDims(_rows(x, sh), dim, sx, 0, _io("x", x), eps, None, 0)


def layer_norm_fwd(x, weight, bias=None, *, eps=1e-5, out=None, stream=None):
    """Layer norm of x's last dimension: (x - mean) / sqrt(var + eps) weight + bias.  weight, bias:
    float32 (dim,), bias may be None; eps: 2^-126 or more.  out may be x.  Returns y, x's shape
    and dtype."""
    import torch

    _device(x, weight, bias, out)
    dims = _layer_dims(x, weight, bias, eps)
    with _on(stream):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            if out.dtype is not x.dtype or out.shape != x.shape:
                raise ValueError("out must have the shape and dtype of x")
            dims.y_stride = _matrix("out", out, out.shape)
        _ok(ssm_layer_norm_fwd(x, weight, bias, out, dims, stream), "ssm_layer_norm_fwd")
    return out


def layer_norm_bwd(x, weight, *, dy, bias=True, eps=1e-5, workspace=None, stream=None) -> dict:
    """Gradients of sum(dy * y) of layer_norm_fwd: dx (x's dtype), dweight and, unless bias is
    False, dbias (float32)."""
    import torch

    _device(x, weight, dy, workspace)
    dims = _layer_dims(x, weight, None, eps)
    _dense("dy", dy, x.dtype, x.shape)
    with _on(stream):
        res = {"dx": torch.empty(x.shape, dtype=x.dtype, device=x.device), "dweight": torch.empty_like(weight)}
        if bias:
            res["dbias"] = torch.empty_like(weight)
        need = ssm_layer_norm_bwd_workspace_bytes(dims)
        workspace, dims.workspace_bytes = _workspace(need, workspace, x.device)
        dims.workspace = _ptr(workspace)
        _ok(ssm_layer_norm_bwd(x, weight, dy, res["dx"], res["dweight"], res.get("dbias"), dims, stream),
            "ssm_layer_norm_bwd")
    return res
