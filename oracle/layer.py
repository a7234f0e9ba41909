"""Float64 oracle of the operators around the scan (test infrastructure, numpy).

Each forward function is the definition written out token by token (or row by
row); each backward function is the chain rule through the same statements in
reverse order.  ``tests/test_oracle_layer_pins.py`` pins the forwards against
closed forms and the backwards against central differences of the forwards.
No code is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    out = np.empty_like(v, dtype=np.float64)
    pos = v >= 0
    out[pos] = 1.0 / (1.0 + np.exp(-v[pos]))
    e = np.exp(v[~pos])
    out[~pos] = e / (1.0 + e)
    return out


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s + v * s * (1.0 - s)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def conv1d(x, weight, bias=None, init=None, pad=None, act=True):
    """x [b,L,D], weight [D,W], init [b,W-1,D].  Returns (y, final)."""
    b, L, D = x.shape
    W = weight.shape[1]
    y, final = np.zeros((b, L, D)), np.zeros((b, W - 1, D))
    for i in range(b):
        p = 0 if pad is None else int(np.clip(pad[i], 0, L))
        seq = [np.zeros(D)] * (W - 1) if init is None else [init[i, j] for j in range(W - 1)]
        for t in range(p, L):
            seq.append(x[i, t])
            v = np.zeros(D) if bias is None else bias.astype(np.float64).copy()
            for k in range(W):
                v = v + weight[:, k] * seq[len(seq) - W + k]
            y[i, t] = silu(v) if act else v
        for j in range(W - 1):
            final[i, j] = seq[len(seq) - (W - 1) + j]
    return y, final


def conv1d_bwd(x, weight, bias, init, dy, dfinal=None, act=True):
    b, L, D = x.shape
    W = weight.shape[1]
    out = {"dx": np.zeros((b, L, D)), "dweight": np.zeros((D, W)), "dbias": np.zeros(D),
           "dinit_state": np.zeros((b, W - 1, D))}
    for i in range(b):
        kept = np.zeros((W - 1, D)) if init is None else init[i]
        seq = np.concatenate([kept, x[i]], 0)
        dseq = np.zeros_like(seq)
        if dfinal is not None:
            dseq[L:] += dfinal[i]
        for t in range(L):
            v = np.zeros(D) if bias is None else bias.astype(np.float64).copy()
            for k in range(W):
                v = v + weight[:, k] * seq[t + k]
            d = dy[i, t] * (dsilu(v) if act else 1.0)
            out["dbias"] += d
            for k in range(W):
                out["dweight"][:, k] += d * seq[t + k]
                dseq[t + k] += d * weight[:, k]
        out["dinit_state"][i], out["dx"][i] = dseq[:W - 1], dseq[W - 1:]
    return out


def _groups(v, D):
    """[b, G, N] -> [b, D, N]: channel d takes group d / (D / G)."""
    return np.repeat(v, D // v.shape[1], axis=1)


def selective_step(h, x, dt_raw, dt_bias, A, B, C, D, z=None):
    """One token: h [b,D,N] before it; x, dt_raw, z [b,D]; B, C [b,G,N].  Returns (h, y)."""
    ch = x.shape[-1]
    dt = softplus(dt_raw + (0.0 if dt_bias is None else dt_bias))
    h = np.exp(dt[..., None] * A) * h + (dt * x)[..., None] * _groups(B, ch)
    y = (h * _groups(C, ch)).sum(-1) + (0.0 if D is None else D * x)
    return h, (y if z is None else y * silu(z))


def selective_scan(x, dt_raw, dt_bias, A, B, C, D, z=None, init=None, pad=None):
    """x, dt_raw, z [b,L,D], A [D,N], B, C [b,L,G,N], init [b,D,N].  Returns (y, final)."""
    b, L, ch = x.shape
    y, final = np.zeros((b, L, ch)), np.zeros((b, ch, A.shape[1]))
    for i in range(b):
        h = np.zeros((1, ch, A.shape[1])) if init is None else init[i:i + 1]
        p = 0 if pad is None else int(np.clip(pad[i], 0, L))
        for t in range(p, L):
            s = slice(i, i + 1)
            h, yt = selective_step(h, x[s, t], dt_raw[s, t], dt_bias, A, B[s, t], C[s, t], D,
                                   None if z is None else z[s, t])
            y[i, t] = yt[0]
        final[i] = h[0]
    return y, final


def selective_scan_bwd(x, dt_raw, dt_bias, A, B, C, D, z, init, dy, dfinal=None):
    b, L, ch = x.shape
    G, N = B.shape[2], B.shape[3]
    zb = dt_raw + (0.0 if dt_bias is None else dt_bias)
    dt = softplus(zb)
    h = np.zeros((b, L + 1, ch, N))
    if init is not None:
        h[:, 0] = init
    for t in range(L):
        h[:, t + 1] = np.exp(dt[:, t, :, None] * A) * h[:, t] + (dt[:, t] * x[:, t])[..., None] * _groups(B[:, t], ch)
    skip = np.zeros(ch) if D is None else D
    gate = np.ones_like(x) if z is None else silu(z)
    out = {"dx": np.zeros_like(x), "ddt_raw": np.zeros_like(x), "dz": None if z is None else np.zeros_like(x),
           "dB": np.zeros_like(B), "dC": np.zeros_like(B), "dA": np.zeros((ch, N)), "ddt_bias": np.zeros(ch),
           "dD": np.zeros(ch)}
    w = np.zeros((b, ch, N)) if dfinal is None else dfinal.copy()
    for t in range(L - 1, -1, -1):
        Bt, Ct = _groups(B[:, t], ch), _groups(C[:, t], ch)
        g = dy[:, t] * gate[:, t]
        w = w + g[..., None] * Ct
        a = np.exp(dt[:, t, :, None] * A)
        carried = w * a * h[:, t]
        wB = (w * Bt).sum(-1)
        out["dx"][:, t] = dt[:, t] * wB + skip * g
        ddt = x[:, t] * wB + (carried * A).sum(-1)
        out["ddt_raw"][:, t] = ddt * sigmoid(zb[:, t])
        out["dC"][:, t] = (h[:, t + 1] * g[..., None]).reshape(b, G, ch // G, N).sum(2)
        out["dB"][:, t] = (w * (dt[:, t] * x[:, t])[..., None]).reshape(b, G, ch // G, N).sum(2)
        out["dA"] += (carried * dt[:, t, :, None]).sum(0)
        out["dD"] += (g * x[:, t]).sum(0)
        if z is not None:
            out["dz"][:, t] = dy[:, t] * ((h[:, t + 1] * Ct).sum(-1) + skip * x[:, t]) * dsilu(z[:, t])
        w = w * a
    out["ddt_bias"] = out["ddt_raw"].sum((0, 1))
    out["dinit_state"] = w
    return out


def group_norm(x, weight, bias, z, ngroups, eps, center, act):
    """x, z [rows, C]; act: "none", "silu", "after", "before"."""
    return _norm(x, weight, bias, z, ngroups, eps, center, act)[0]


def _norm(x, weight, bias, z, ngroups, eps, center, act):
    rows, C = x.shape
    u = (x * silu(z) if act == "before" else x).reshape(rows, ngroups, C // ngroups)
    c = u - u.mean(-1, keepdims=True) if center else u
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    n = (c * r).reshape(rows, C)
    v = n * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    y = silu(v) if act == "silu" else v * silu(z) if act == "after" else v
    return y, n, v, r


def group_norm_bwd(x, weight, bias, z, dy, ngroups, eps, center, act):
    rows, C = x.shape
    _, n, v, r = _norm(x, weight, bias, z, ngroups, eps, center, act)
    dz, dv = None, dy
    if act == "silu":
        dv = dy * dsilu(v)
    elif act == "after":
        dz, dv = dy * v * dsilu(z), dy * silu(z)
    shape = (rows, ngroups, C // ngroups)
    dn, ng = (dv * (1.0 if weight is None else weight)).reshape(shape), n.reshape(shape)
    du = dn - ng * (dn * ng).mean(-1, keepdims=True)
    if center:
        du = du - dn.mean(-1, keepdims=True)
    dx = (du * r).reshape(rows, C)
    if act == "before":
        dx, dz = dx * silu(z), dx * x * dsilu(z)
    return {"dx": dx, "dz": dz, "dweight": (dv * n).sum(0), "dbias": dv.sum(0)}
