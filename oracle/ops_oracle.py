"""64-bit definitions of the operators around the routed layer: the norm with
the residual's addition, tokens sorted by expert and back with their weights,
the router's gradient, and the gradients of the others.

Plain numpy in float64, written from the formulas; no rounding to a stored type
anywhere.  Test infrastructure.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100


def rmsnorm(x, weight, eps, residual=None):
    """(r, y): r = x + residual, y = r * weight / sqrt(mean r^2 + eps)."""
    r = np.asarray(x, np.float64)
    if residual is not None:
        r = r + np.asarray(residual, np.float64)
    rms = np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    return r, r / rms * np.asarray(weight, np.float64)


def e4m3_scales(y, group):
    """Scales [T][groups] of an 8-bit output (group 0: one a row)."""
    T, H = y.shape
    g = group if group else H
    return np.stack([np.maximum(np.abs(y[:, i:i + g]).max(axis=1) / E4M3_MAX, SCALE_MIN) for i in range(0, H, g)],
                    axis=1)


def rmsnorm_backward(dy, r, weight, eps, dresidual=None):
    """(dx, dweight) of y = r weight / sqrt(mean r^2 + eps)."""
    dy, r, g = (np.asarray(a, np.float64) for a in (dy, r, weight))
    H = r.shape[1]
    s = 1 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    d = np.sum(g * dy * r, axis=1, keepdims=True)
    dx = s * g * dy - r * s ** 3 * d / H
    if dresidual is not None:
        dx = dx + np.asarray(dresidual, np.float64)
    return dx, np.sum(dy * r * s, axis=0)


def sort_slots(ids, E):
    """(offsets [E+1], inv [S], perm [kept]) of ids [T][k]; a dropped slot has inv -1."""
    flat = np.asarray(ids).reshape(-1)
    perm = np.array([s for e in range(E) for s in np.nonzero(flat == e)[0]], dtype=np.int64)
    inv = np.full(flat.shape, -1, np.int64)
    inv[perm] = np.arange(len(perm))
    offsets = np.concatenate([[0], np.cumsum([np.sum(flat == e) for e in range(E)])])
    return offsets, inv, perm


def unpermute(rows, inv, w, T, k):
    """y[t] = sum_j w[t][j] rows[inv[t k + j]]; w None: ones."""
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            p = inv[t * k + j]
            if p >= 0:
                y[t] += (1.0 if w is None else float(w[t, j])) * rows[p].astype(np.float64)
    return y


def unpermute_backward(dy, rows, inv, w, T, k):
    """(drows, dw); rows without a slot are zero."""
    drows = np.zeros((T * k, dy.shape[1]))
    dw = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = inv[t * k + j]
            if p >= 0:
                drows[p] = (1.0 if w is None else float(w[t, j])) * dy[t].astype(np.float64)
                dw[t, j] = float(np.dot(dy[t].astype(np.float64), rows[p].astype(np.float64)))
    return drows, dw


def router_backward(x, router_w, ids, w, dw, dx_add=None):
    """(dx, drouter_w) of w = softmax over the selected logits <x, router_w[ids]>."""
    x, router_w, w, dw = (np.asarray(a, np.float64) for a in (x, router_w, w, dw))
    E = router_w.shape[0]
    T, k = ids.shape
    dx = np.zeros_like(x) if dx_add is None else np.asarray(dx_add, np.float64).copy()
    drouter = np.zeros_like(router_w)
    for t in range(T):
        kept = [j for j in range(k) if 0 <= ids[t, j] < E]
        mean = sum(w[t, j] * dw[t, j] for j in kept)
        for j in kept:
            dl = w[t, j] * (dw[t, j] - mean)
            dx[t] += dl * router_w[ids[t, j]]
            drouter[ids[t, j]] += dl * x[t]
    return dx, drouter
