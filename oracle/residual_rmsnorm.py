"""Plain float64 oracle of the residual step between two blocks (test infrastructure only).

Only ``tests/`` may import this module.  Written from the definition in
include/residual_rmsnorm.h; ``gate`` is None, [n] or [m, n].
"""
from __future__ import annotations

import numpy as np

E32 = 2.0 ** -24


def _gate(gate, shape):
    return np.ones(shape) if gate is None else np.broadcast_to(gate, shape)


def forward(f, x, gate, w_post, w_pre, eps: float, scale: float):
    """(H, Y, rstd) in float64."""
    rp = 1 / np.sqrt((f * f).mean(1) + eps)
    h = x + scale * _gate(gate, f.shape) * (f * rp[:, None] * w_post)
    rq = 1 / np.sqrt((h * h).mean(1) + eps)
    return h, h * rq[:, None] * w_pre, np.stack([rp, rq], 1)


def backward(f, h, gate, w_post, w_pre, rstd, dy, dh, scale: float):
    """(dF, dX, dgate, dW_post, dW_pre): dgate is [m, n] here, before any sum over rows."""
    n = f.shape[1]
    rp, rq = rstd[:, :1], rstd[:, 1:]
    g = rq * (w_pre * dy - h * rq ** 2 * (w_pre * dy * h).sum(1, keepdims=True) / n)
    if dh is not None:
        g = g + dh
    z = f * rp * w_post
    dz = scale * g * _gate(gate, f.shape)
    df = rp * (w_post * dz - f * rp ** 2 * (w_post * dz * f).sum(1, keepdims=True) / n)
    return df, g, scale * g * z, (dz * f * rp).sum(0), (dy * h * rq).sum(0)


def forward_bounds(f, x, gate, w_post, w_pre, eps, scale, out, tiny):
    """Element-wise bounds: a float32 sum of n terms rounds each partial sum once (n e relative for squares, halved by
    the square root), every product and quotient once more, and the result to the output type."""
    n = f.shape[1]
    h, y, rstd = forward(f, x, gate, w_post, w_pre, eps, scale)
    rel = (n + 16) * E32
    branch = np.abs(scale * _gate(gate, f.shape) * f * rstd[:, :1] * w_post)
    eh = rel * branch + 4 * E32 * (np.abs(x) + branch)
    erq = rel + (np.abs(h) * eh).sum(1) / np.maximum((h * h).sum(1) + n * eps, 1e-300)
    return (eh + out * np.abs(h) + tiny,
            (eh * rstd[:, 1:] + erq[:, None] * np.abs(h) * rstd[:, 1:]) * np.abs(w_pre) * 2 + out * np.abs(y) + tiny,
            np.stack([rel * rstd[:, 0], erq * rstd[:, 1]], 1))


def backward_bounds(f, h, gate, w_post, w_pre, rstd, dy, dh, scale, out, tiny):
    """Bounds of backward()'s results, the same way; the sums over m rows add m e of the terms' magnitudes."""
    m, n = f.shape
    rp, rq = rstd[:, :1], rstd[:, 1:]
    e, gt = E32, np.abs(_gate(gate, f.shape))
    wy = np.abs(w_pre * dy)
    eg = rq * ((n + 16) * e * np.abs(h) * rq ** 2 * (wy * np.abs(h)).sum(1, keepdims=True) / n + 8 * e * wy)
    if dh is not None:
        eg = eg + 4 * e * np.abs(dh)
    df, g, dgate, dw_post, dw_pre = backward(f, h, gate, w_post, w_pre, rstd, dy, dh, scale)
    eg = eg + 4 * e * np.abs(g)
    s = abs(scale)
    edz = s * gt * eg + 8 * e * s * gt * np.abs(g)
    wz = np.abs(w_post) * (s * gt * np.abs(g))
    inner = (np.abs(w_post) * edz * np.abs(f)).sum(1, keepdims=True) / n \
        + (n + 16) * e * (wz * np.abs(f)).sum(1, keepdims=True) / n
    edf = rp * (np.abs(w_post) * edz + np.abs(f) * rp ** 2 * inner) + 8 * e * rp * wz \
        + 8 * e * np.abs(f) * rp ** 3 * (wz * np.abs(f)).sum(1, keepdims=True) / n
    z = np.abs(f * rp * w_post)
    edg = s * eg * z + 8 * e * s * np.abs(g) * z
    epost = (edz * np.abs(f) * rp).sum(0) + (m + 16) * e * (s * gt * np.abs(g) * np.abs(f) * rp).sum(0)
    epre = (m + 16) * e * (np.abs(dy * h) * rq).sum(0)
    return {"df": edf + out * np.abs(df) + tiny, "dx": eg + out * np.abs(g) + tiny,
            "dgate": edg + out * np.abs(dgate) + tiny,
            "dgate_sum": edg.sum(0) + (m + 16) * e * np.abs(dgate).sum(0), "dw_post": epost, "dw_pre": epre}
