"""Plain float64 reference of the gated delta rule and of the layer norm: token by token, row by
row, with the gradients of the recurrence itself."""
import numpy as np


def _spread(x, heads):
    return np.repeat(x, heads // x.shape[1], 1)


def delta(q, k, v, g, beta, scale, starts, s0=None):
    """q, k (T, Hk, dk), v (T, H, dv), g, beta (T, H); starts: cumulative lengths.  Returns o
    (zero in rows of no sequence) and the final states (nseq, H, dk, dv)."""
    T, H, dv = v.shape
    dk, n = q.shape[2], len(starts) - 1
    q, k, a = _spread(q, H), _spread(k, H), np.exp(np.maximum(g, -128.0))
    o, last = np.zeros((T, H, dv)), np.zeros((n, H, dk, dv))
    for s in range(n):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[s].astype(np.float64)
        for t in range(starts[s], starts[s + 1]):
            S = S * a[t][:, None, None]
            r = v[t] - np.einsum("hkv,hk->hv", S, k[t])
            S = S + k[t][:, :, None] * (beta[t][:, None] * r)[:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        last[s] = S
    return o, last


def delta_grads(q, k, v, g, beta, scale, starts, do, s0=None, ds_last=None):
    """dq, dk (per shared head), dv, dg (T, H), dbeta, ds0."""
    T, H, dv = v.shape
    Hk, dk = q.shape[1:]
    n = len(starts) - 1
    qr, kr, a = _spread(q, H), _spread(k, H), np.exp(np.maximum(g, -128.0))
    dq, dkk, dvv = np.zeros((T, H, dk)), np.zeros((T, H, dk)), np.zeros((T, H, dv))
    dg, db, ds0 = np.zeros((T, H)), np.zeros((T, H)), np.zeros((n, H, dk, dv))
    for s in range(n):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[s].astype(np.float64)
        kept = {}
        for t in range(starts[s], starts[s + 1]):
            Sp = S * a[t][:, None, None]
            r = v[t] - np.einsum("hkv,hk->hv", Sp, kr[t])
            S = Sp + kr[t][:, :, None] * (beta[t][:, None] * r)[:, None, :]
            kept[t] = Sp, r, S
        dS = np.zeros((H, dk, dv)) if ds_last is None else ds_last[s].astype(np.float64)
        for t in range(starts[s + 1] - 1, starts[s] - 1, -1):
            Sp, r, S = kept[t]
            dq[t] = scale * np.einsum("hkv,hv->hk", S, do[t])
            dS = dS + scale * qr[t][:, :, None] * do[t][:, None, :]
            du = np.einsum("hkv,hk->hv", dS, kr[t])
            db[t] = (du * r).sum(-1)
            dr = beta[t][:, None] * du
            dvv[t] = dr
            dkk[t] = np.einsum("hkv,hv->hk", dS, beta[t][:, None] * r) - np.einsum("hkv,hv->hk", Sp, dr)
            dS = dS - kr[t][:, :, None] * dr[:, None, :]
            dg[t] = (dS * Sp).sum((1, 2))
            dS = dS * a[t][:, None, None]
        ds0[s] = dS
    fold = lambda x: x.reshape(T, Hk, H // Hk, dk).sum(2)   # noqa: E731
    return dict(dq=fold(dq), dk=fold(dkk), dv=dvv, dg=dg, dbeta=db, ds0=ds0)


def layer_norm(x, w, b, eps):
    d = x - x.mean(-1, keepdims=True)
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps) * w
    return y if b is None else y + b


def layer_norm_grads(x, w, dy, eps):
    d = x - x.mean(-1, keepdims=True)
    r = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n, up = d * r, dy * w
    dx = r * (up - up.mean(-1, keepdims=True) - n * (up * n).mean(-1, keepdims=True))
    return dict(dx=dx, dweight=(dy * n).sum(0), dbias=dy.sum(0))
