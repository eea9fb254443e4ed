"""fp64 reference of the operators around the layer: the block norms and their
gradients, the grouped products, and the AdamW step with 32-bit or 8-bit
moments.  Plain numpy, written from the formulas; shares nothing with the CUDA
path."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- block norms
def inv_rms(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def norm(x, w, eps):
    return x * inv_rms(x, eps) * w


def gate_rows(gate, gate_group, T):
    """[T, d]: the gate of every token (ones without a gate)."""
    if gate is None:
        return 1.0
    return gate[np.arange(T) // gate_group]


def combine_norm(u, y_slots, w, gate, gate_group, res_scale, w_next, eps):
    """(h, y, x_next) of one block end; y_slots [T, S, d]."""
    y = y_slots.sum(axis=1)
    h = res_scale * u + gate_rows(gate, gate_group, len(u)) * norm(y, w, eps)
    return h, y, None if w_next is None else norm(h, w_next, eps)


def _through_norm(v, c, eps):
    r = inv_rms(v, eps)
    return r * c - v * r ** 3 * np.mean(v * c, axis=-1, keepdims=True)


def norm_backward(x, w, dout, dh, res_scale, eps):
    """(dx, dw) of x -> norm(x) w, the residual's gradient res_scale * dh added."""
    dx = _through_norm(x, dout * w, eps)
    if dh is not None:
        dx = dx + res_scale * dh
    return dx, np.sum(dout * x * inv_rms(x, eps), axis=0)


def combine_norm_backward(y, w, gate, gate_group, dh, eps):
    """(dy, dw, dgate) of h = res u + gate * (norm(y) w)."""
    T = len(y)
    g = gate_rows(gate, gate_group, T)
    n = y * inv_rms(y, eps)
    dgate = None
    if gate is not None:
        dgate = np.zeros_like(gate)
        np.add.at(dgate, np.arange(T) // gate_group, dh * w * n)
    return _through_norm(y, dh * g * w, eps), np.sum(dh * g * n, axis=0), dgate


# ---------------------------------------------------------------- grouped products
def _groups(offsets):
    """(group, its rows); a group whose offsets decrease is empty."""
    return [(g, slice(a, b)) for g, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])) if b > a]


def grouped_mm(x, w, offsets, y):
    """y[r] = w[g] x[r]; rows of no group keep what y holds."""
    y = y.copy()
    for g, r in _groups(offsets):
        y[r] = x[r] @ w[g].T
    return y


def grouped_mm_dx(dy, w, offsets, dx):
    return grouped_mm(dy, w.transpose(0, 2, 1), offsets, dx)


def grouped_mm_dw(dy, x, offsets, dw):
    """dw[g] + sum_r dy[r] x[r]^T."""
    dw = dw.copy()
    for g, r in _groups(offsets):
        dw[g] += dy[r].T @ x[r]
    return dw
