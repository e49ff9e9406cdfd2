"""fp64 reference of the mixture-of-experts operators: the RMS norm with the residual's addition
(and its 8-bit output), sorting by expert, dispatch, combine, the experts' products, the layer
they form, and every gradient.

TEST INFRASTRUCTURE ONLY: numpy loops and products, nothing shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def f64(a):
    return np.asarray(a, np.float64)


def rms_norm(x, residual, weight, eps):
    """(y, h, rstd)."""
    h = f64(x) if residual is None else f64(x) + f64(residual)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    y = h * rstd[:, None]
    return (y if weight is None else y * f64(weight)), h, rstd


def e4m3_scales(y, group):
    """[rows, groups]: max|y| / 448 over each group of columns (group 0: the row)."""
    width = y.shape[1]
    group = group or width
    return np.stack([np.abs(y[:, c:c + group]).max(axis=1)
                     for c in range(0, width, group)], axis=1) / 448.0


def rms_norm_bwd(dy, h, rstd, weight, dsum):
    """(dx, dweight) at the stored h and rstd."""
    xh = f64(h) * f64(rstd)[:, None]
    g = f64(dy) if weight is None else f64(dy) * f64(weight)
    dx = f64(rstd)[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + f64(dsum)
    return dx, (f64(dy) * xh).sum(axis=0)


def sort(ids, experts):
    """(slots, offsets, rows): pairs in order of (expert, pair number)."""
    T, k = ids.shape
    slots = np.full(T * k, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int64)
    rows = []
    for e in range(experts):
        for p in np.flatnonzero(ids.reshape(-1) == e):
            slots[p] = len(rows)
            rows.append(p // k)
        offsets[e + 1] = len(rows)
    return slots.reshape(T, k), offsets, np.asarray(rows, np.int64)


def combine(y, slots, weights, residual):
    T, k = slots.shape
    out = np.zeros((T, y.shape[1])) if residual is None else f64(residual).copy()
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                out[t] += (1.0 if weights is None else float(weights[t, j])) * f64(y[slots[t, j]])
    return out


def combine_bwd(dout, y, slots, weights):
    """(dy with zeros in rows that no slot names, dweights)."""
    T, k = slots.shape
    dy, dw = np.zeros(y.shape), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            s = slots[t, j]
            if s >= 0:
                dy[s] = (1.0 if weights is None else float(weights[t, j])) * f64(dout[t])
                dw[t, j] = f64(dout[t]) @ f64(y[s])
    return dy, dw


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def silu_slope(x):
    with np.errstate(over="ignore"):
        p = 1.0 / (1.0 + np.exp(-x))
    return p * (1.0 + x * (1.0 - p))


def proj(x, w, offsets):
    """[rows, d_out], zeros in rows of no expert; w [experts, d_in, d_out]."""
    out = np.zeros((x.shape[0], w.shape[2]))
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        out[a:b] = f64(x[a:b]) @ f64(w[e])
    return out


def proj_bwd(dout, x, w, offsets, silu_pre=None):
    """(dx, dw)."""
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        dx[a:b] = f64(dout[a:b]) @ f64(w[e]).T
        dw[e] = f64(x[a:b]).T @ f64(dout[a:b])
    if silu_pre is not None:
        dx *= silu_slope(f64(silu_pre))
    return dx, dw


def layer(x, residual, norm_weight, ids, gates, w_in, w_out, eps):
    """The layer's output and what its backward needs."""
    n, h, rstd = rms_norm(x, residual, norm_weight, eps)
    slots, offsets, rows = sort(ids, w_in.shape[0])
    xs = n[rows]
    pre = proj(xs, w_in, offsets)
    z = silu(pre)
    y = proj(z, w_out, offsets)
    return dict(o=combine(y, slots, gates, h), h=h, rstd=rstd, slots=slots, offsets=offsets,
                rows=rows, xs=xs, pre=pre, z=z, y=y)


def layer_bwd(do, s, norm_weight, gates, w_in, w_out):
    dy, dgates = combine_bwd(do, s["y"], s["slots"], gates)
    dpre, dw_out = proj_bwd(dy, s["z"], w_out, s["offsets"], s["pre"])
    dxs, dw_in = proj_bwd(dpre, s["xs"], w_in, s["offsets"])
    dn = combine(dxs, s["slots"], None, None) if len(dxs) else np.zeros(do.shape)
    dx, dnw = rms_norm_bwd(dn, s["h"], s["rstd"], norm_weight, do)
    return dict(dx=dx, dnorm_weight=dnw, dgates=dgates, dw_in=dw_in, dw_out=dw_out)
