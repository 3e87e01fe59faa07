"""Plain float64 references of the block operators (token by token, row by row), and the
magnitudes that their error bounds are stated in.

``linattn``/``linattn_grads`` walk the recurrence one token at a time.  Run on the absolute
values of the inputs they give, for every output, the sum of the absolute values of its
terms: rounding errors are bounded by a small multiple of that sum.
"""
import numpy as np


def linattn(q, k, v, g, scale, starts, s0=None):
    """q, k (T, Hk, dk), v (T, H, dv), g (T, H); starts: cumulative lengths.  Returns o
    (zero in rows of no sequence) and the final states (nseq, H, dk, dv)."""
    T, H, dv = v.shape
    dk, rep = q.shape[2], H // q.shape[1]
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    n = len(starts) - 1
    o = np.zeros((T, H, dv))
    last = np.zeros((n, H, dk, dv))
    for s in range(n):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[s].astype(np.float64)
        for t in range(starts[s], starts[s + 1]):
            S = S * np.exp(np.maximum(g[t], -128.0))[:, None, None] + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        last[s] = S
    return o, last


def linattn_grads(q, k, v, g, scale, starts, do, s0=None, ds_last=None):
    """dq, dk (per shared head), dv, dg (T, H), ds0."""
    T, H, dv = v.shape
    Hk, dk = q.shape[1:]
    rep = H // Hk
    qr, kr = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    g = np.maximum(g, -128.0)
    n = len(starts) - 1
    dq, dkk, dvv, dg = np.zeros((T, H, dk)), np.zeros((T, H, dk)), np.zeros((T, H, dv)), np.zeros((T, H))
    ds0 = np.zeros((n, H, dk, dv))
    for s in range(n):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[s].astype(np.float64)
        before = {}
        for t in range(starts[s], starts[s + 1]):
            before[t] = S
            S = S * np.exp(g[t])[:, None, None] + kr[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hkv,hv->hk", S, do[t])
        R = np.zeros((H, dk, dv)) if ds_last is None else ds_last[s].astype(np.float64)
        for t in range(starts[s + 1] - 1, starts[s] - 1, -1):
            R = R + scale * qr[t][:, :, None] * do[t][:, None, :]
            dkk[t] = np.einsum("hkv,hv->hk", R, v[t])
            dvv[t] = np.einsum("hkv,hk->hv", R, kr[t])
            dg[t] = np.exp(g[t]) * np.einsum("hkv,hkv->h", before[t], R)
            R = R * np.exp(g[t])[:, None, None]
        ds0[s] = R
    fold = lambda x: x.reshape(T, Hk, rep, dk).sum(2)   # noqa: E731
    return dict(dq=fold(dq), dk=fold(dkk), dv=dvv, dg=dg, ds0=ds0)


def silu(z):
    return z / (1 + np.exp(-z))


def rms(x, eps):
    return 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def gated_norm(x, z, w, group, first, eps):
    """x, z (rows, dim); w (dim,) or (group,)."""
    rows, dim = x.shape
    x = x.reshape(rows, -1, group)
    a = np.ones_like(x) if z is None else silu(z.reshape(x.shape))
    w = np.broadcast_to(w.reshape(-1, group), x.shape[1:])
    p = x * a if first else x
    y = p * rms(p, eps) * w
    return (y if first else y * a).reshape(rows, dim)


def rms_grad(dn, x, eps):
    """Gradient at x of sum(dn * x * rms(x))."""
    r = rms(x, eps)
    n = x * r
    return r * (dn - n * (dn * n).mean(-1, keepdims=True))


def gated_norm_grads(x, z, w, dy, group, first, eps):
    rows, dim = x.shape
    shape = (rows, dim // group, group)
    x, dy = x.reshape(shape), dy.reshape(shape)
    zz = np.zeros(shape) if z is None else z.reshape(shape)
    sg = 1 / (1 + np.exp(-zz))
    a = np.ones(shape) if z is None else zz * sg
    da = sg * (1 + zz * (1 - sg))
    wf = np.broadcast_to(w.reshape(-1, group), shape[1:])
    p = x * a if first else x
    n = p * rms(p, eps)
    up = dy if first else dy * a
    dp = rms_grad(up * wf, p, eps)
    dw = (up * n).sum(0)
    if w.size == group and dim != group:
        dw = dw.sum(0)
    out = dict(dx=(dp * a if first else dp).reshape(rows, dim), dweight=dw.reshape(-1))
    if z is not None:
        out["dz"] = ((dp * x if first else dy * n * wf) * da).reshape(rows, dim)
    return out


def add_norm(x, res, w, scale, post, eps, store):
    """Returns (y, r before it is stored, r as stored); ``store`` rounds r."""
    a = x if post is None else x * rms(x, eps) * post
    r = (0.0 if res is None else res) + (a if scale is None else scale * a)
    f = store(r)
    return f * rms(f, eps) * w, r, f


def add_norm_grads(x, r, w, dy, dr, scale, post, eps):
    out = dict(dweight=(dy * r * rms(r, eps)).sum(0))
    d = rms_grad(dy * w, r, eps) + (0.0 if dr is None else dr)
    out["dresidual"] = d
    n = x * rms(x, eps) if post is not None else x
    if scale is not None:
        out["dscale"] = (d * (n * post if post is not None else n)).sum(0)
        d = d * scale
    if post is not None:
        out["dpost_weight"] = (d * n).sum(0)
        d = rms_grad(d * post, x, eps)
    out["dx"] = d
    return out
