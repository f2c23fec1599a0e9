"""Plain float64 oracle of causal attention over packed sequences (test infrastructure only).

Only ``tests/`` and ``__graft_entry__.smoke()`` may import this module; the CUDA
library never links, loads or calls it.  Everything is written from the
definition in include/mha_packed.h, one sequence and one head at a time, with
numpy matrix products in float64.  A term that a query does not attend is left
out by selection, never multiplied by zero.

Beside each result stands what a float32 implementation may be off, element by
element (``forward_bounds``, ``backward_bounds``), from first-order error terms:
with e = 2^-24 (float32's unit roundoff), u the input type's (2^-8 bf16, 2^-11
fp16, 0 for float32) where an implementation rounds P and dS, and out the output
type's,
  * a score of d products is off by at most E = (d + 4) e sum |q||k| / sqrt(d)
    (each product and sum rounds once), so exp of it by a relative E;
  * a sum of n terms rounds each partial sum once: n e times the terms' magnitudes;
  * the exponential, the division and the logarithm add a few roundings: 8 e in
    relative terms, and the statistics folded into one float32 exponent add
    (|m| + |l|) 4 e.
"""
from __future__ import annotations

import numpy as np

E32 = 2.0 ** -24


def sequences(offsets):
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:]) if b > a]


def attended(n: int, window: int) -> np.ndarray:
    """[query, key]: t <= pos and (no window or pos < t + window)."""
    pos = np.arange(n)
    keep = pos[None, :] <= pos[:, None]
    return keep & (pos[:, None] < pos[None, :] + window) if window else keep


def _masked_dot(w, x, keep):
    """sum over t of w[pos, t] x[t], over the attended t only (w is 0 elsewhere, x may hold infinities or NaN there)."""
    if np.isfinite(x).all():
        return w @ x
    out = np.zeros((w.shape[0], x.shape[1]))
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(w.shape[0]):
            out[i] = (w[i, keep[i], None] * x[keep[i]]).sum(0)
    return out


def forward(q, k, v, offsets, window: int):
    """O [T, H, d] and LSE [T, H, 2] in float64."""
    T, H, d = q.shape
    per = H // k.shape[1]
    o, lse = np.zeros((T, H, d)), np.zeros((T, H, 2))
    lse[..., 1] = np.inf
    for a, b in sequences(offsets):
        keep = attended(b - a, window)
        for h in range(H):
            with np.errstate(invalid="ignore"):
                s = np.where(keep, (q[a:b, h] @ k[a:b, h // per].T) / np.sqrt(d), -np.inf)
            m = s.max(1)
            p = np.where(keep, np.exp(s - m[:, None]), 0.0)
            total = p.sum(1)
            o[a:b, h] = _masked_dot(p, v[a:b, h // per], keep) / total[:, None]
            lse[a:b, h, 0], lse[a:b, h, 1] = m, np.log(total)
    return o, lse


def _score_error(x, y, d, scale):
    return (d + 4) * E32 * (np.abs(x) @ np.abs(y).T) * scale


def forward_bounds(q, k, v, offsets, window: int, u: float, out: float, tiny: float):
    """(bound on O, bound on LSE) [T, H, d] and [T, H, 2]; ``tiny``: half the output type's smallest step."""
    T, H, d = q.shape
    per = H // k.shape[1]
    o, lse = forward(q, k, v, offsets, window)
    bo, bl = np.zeros((T, H, d)), np.zeros((T, H, 2))
    for a, b in sequences(offsets):
        keep, n = attended(b - a, window), b - a
        for h in range(H):
            g = h // per
            err = np.where(keep, _score_error(q[a:b, h], k[a:b, g], d, 1 / np.sqrt(d)), 0.0).max(1)
            s = (q[a:b, h] @ k[a:b, g].T) / np.sqrt(d)
            p = np.where(keep, np.exp(s - lse[a:b, h, :1] - lse[a:b, h, 1:]), 0.0)
            rel = 2 * err + (n + 8) * 2 * E32
            bo[a:b, h] = (rel + u)[:, None] * (p @ np.abs(v[a:b, g])) + out * np.abs(o[a:b, h]) + tiny
            bl[a:b, h, 0] = err + 4 * E32 * np.abs(lse[a:b, h, 0])
            bl[a:b, h, 1] = rel + 4 * E32 * (np.abs(lse[a:b, h, 0]) + np.abs(lse[a:b, h, 1]))
    return bo, bl


def backward(q, k, v, o, d_out, lse, offsets, window: int):
    """dQ [T, H, d], dK and dV [T, G, d] in float64, from the given O and LSE."""
    T, H, d = q.shape
    per = H // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        for a, b in sequences(offsets):
            keep = attended(b - a, window)
            for h in range(H):
                g = h // per
                s = (q[a:b, h] @ k[a:b, g].T) / np.sqrt(d)
                p = np.where(keep, np.exp(s - lse[a:b, h, :1] - lse[a:b, h, 1:]), 0.0)
                delta = (d_out[a:b, h] * o[a:b, h]).sum(1, keepdims=True)
                ds = np.where(keep, p * (d_out[a:b, h] @ v[a:b, g].T - delta), 0.0)
                dq[a:b, h] = _masked_dot(ds, k[a:b, g], keep) / np.sqrt(d)
                dk[a:b, g] += _masked_dot(ds.T, q[a:b, h], keep.T) / np.sqrt(d)
                dv[a:b, g] += _masked_dot(p.T, d_out[a:b, h], keep.T)
    return dq, dk, dv


def backward_bounds(q, k, v, o, d_out, lse, offsets, window: int, u: float, out: float, tiny: float):
    """Element-wise bounds of the three gradients."""
    T, H, d = q.shape
    per = H // k.shape[1]
    exact = backward(q, k, v, o, d_out, lse, offsets, window)
    bq, bk, bv = (np.zeros(x.shape) for x in exact)
    for a, b in sequences(offsets):
        keep, n = attended(b - a, window), b - a
        for h in range(H):
            g = h // per
            s = (q[a:b, h] @ k[a:b, g].T) / np.sqrt(d)
            p = np.where(keep, np.exp(s - lse[a:b, h, :1] - lse[a:b, h, 1:]), 0.0)
            delta = (d_out[a:b, h] * o[a:b, h]).sum(1, keepdims=True)
            ds = np.abs(p * (d_out[a:b, h] @ v[a:b, g].T - delta))
            rel = _score_error(q[a:b, h], k[a:b, g], d, 1 / np.sqrt(d)) + 8 * E32 \
                + 4 * E32 * np.abs(lse[a:b, h]).sum(1, keepdims=True)
            add = _score_error(d_out[a:b, h], v[a:b, g], d, 1.0) \
                + (d + 4) * E32 * (np.abs(d_out[a:b, h]) * np.abs(o[a:b, h])).sum(1, keepdims=True)
            tail = u + (n * per + 8) * 2 * E32
            es = (rel + tail) * ds + p * add
            bq[a:b, h] += es @ np.abs(k[a:b, g]) / np.sqrt(d)
            bk[a:b, g] += es.T @ np.abs(q[a:b, h]) / np.sqrt(d)
            bv[a:b, g] += ((rel + tail) * p).T @ np.abs(d_out[a:b, h])
    return tuple(x + out * np.abs(e) + tiny for x, e in zip((bq, bk, bv), exact))
