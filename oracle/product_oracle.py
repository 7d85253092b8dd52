"""64-bit definitions of the experts' products in 16 bits: the product with bias,
activation and residual, the gated feed-forward block, and their gradients.

Plain numpy in float64, one expert after another, written from the formulas; no
rounding to a stored type anywhere.  Test infrastructure.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100

_erfc = np.vectorize(math.erfc, otypes=[np.float64])   # Phi(z) = erfc(-z / sqrt 2) / 2 keeps its digits far below 0


def act(z, name):
    if name == "silu":
        return z / (1 + np.exp(-z))
    if name == "gelu":
        return z * _erfc(-z / math.sqrt(2)) / 2
    return z


def slope(z, name):
    if name == "silu":
        q = 1 / (1 + np.exp(-z))
        return q + z * q * (1 - q)
    if name == "gelu":
        return _erfc(-z / math.sqrt(2)) / 2 + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(z)


def spans(offsets, S, E):
    """(expert, slice of its rows)."""
    ends = [0, S] if offsets is None else [int(v) for v in offsets]
    return [(e, slice(ends[e], ends[e + 1])) for e in range(E)]


def product(x, w, offsets=None, bias=None, name="none", residual=None):
    """(z, y) of z = x w^T + bias, y = act(z) + residual; NaN in rows of no expert."""
    E, N, _ = w.shape
    z = np.full((x.shape[0], N), np.nan)
    for e, at in spans(offsets, len(x), E):
        z[at] = x[at] @ w[e].T + (0 if bias is None else bias[e])
    return z, act(z, name) + (0 if residual is None else residual)


def product_backward(dy, x, w, offsets=None, name="none", pre=None):
    """(dx, dw, dbias, dz)."""
    E, N, K = w.shape
    dx, dw, db = np.full((len(dy), K), np.nan), np.zeros_like(w), np.zeros((E, N))
    dz = dy if name == "none" else dy * slope(pre, name)
    for e, at in spans(offsets, len(dy), E):
        dx[at], dw[e], db[e] = dz[at] @ w[e], dz[at].T @ x[at], dz[at].sum(0)
    return dx, dw, db, dz


def ffn(x, w_gate_up, w_down, offsets=None, name="silu"):
    """(z, h, y) of z = [gate | up], h = act(gate) up, y = h w_down^T."""
    z, _ = product(x, w_gate_up, offsets)
    I = z.shape[1] // 2
    h = act(z[:, :I], name) * z[:, I:]
    return z, h, product(h, w_down, offsets)[0]


def ffn_backward(dy, x, w_gate_up, w_down, z, offsets=None, name="silu"):
    """(dx, dw_gate_up, dw_down, dh)."""
    I = z.shape[1] // 2
    gate, up = z[:, :I], z[:, I:]
    dh, dw_down, _, _ = product_backward(dy, act(gate, name) * up, w_down, offsets)
    dz = np.concatenate([dh * up * slope(gate, name), dh * act(gate, name)], axis=1)
    dx, dw_gate_up, _, _ = product_backward(dz, x, w_gate_up, offsets)
    return dx, dw_gate_up, dw_down, dh


def scales(z):
    """Scales [S][2 G] of the 8-bit checkpoint of z [S][2I]."""
    I = z.shape[1] // 2
    pieces = [z[:, h * I + i:min(h * I + i + GROUP, h * I + I)] for h in (0, 1) for i in range(0, I, GROUP)]
    return np.stack([np.maximum(np.abs(p).max(axis=1) / E4M3_MAX, SCALE_MIN) for p in pieces], axis=1)


def spread_scales(scale, I):
    """The scale of every column: [S][2I]."""
    G = scale.shape[1] // 2
    wide = np.repeat(scale.reshape(len(scale), 2, G), GROUP, axis=2)[:, :, :I]
    return wide.reshape(len(scale), 2 * I)
