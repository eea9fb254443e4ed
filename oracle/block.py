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


# ---------------------------------------------------------------- AdamW
SCALE_BLOCK = 128


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay):
    """(p, m, v) after one step; fp64 arrays."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    root = np.sqrt(v / (1 - beta2 ** step))
    return p - lr * (decay * p + m / (1 - beta1 ** step) / (root + eps)), m, v


def block_scales(x):
    """max |x| / 448 of every 128 elements, the last block short."""
    pad = np.concatenate([x, np.zeros(-len(x) % SCALE_BLOCK)])
    return np.abs(pad).reshape(-1, SCALE_BLOCK).max(1) / 448.0


def spread(scales, n):
    return np.repeat(scales, SCALE_BLOCK)[:n]


def e4m3_value(codes):
    """Values of E4M3 codes (uint8)."""
    c = codes.astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e > 0, (8 + f) * 2.0 ** (e - 10), f * 2.0 ** -9)
    mag = np.where((c & 0x7f) == 0x7f, np.nan, mag)
    return np.where(c & 0x80, -mag, mag)


def e4m3_position(a):
    """Place of magnitudes 0 <= a <= 448 on the scale of the codes: a whole number at a code's
    value, linear between two codes."""
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -40))), -6)
    return np.where(a < 2.0 ** -6, a * 512, (e + 7) * 8 + (a / 2.0 ** e - 1) * 8)


def random_words(n, tensor, seed, step):
    """The generator's 32 bits for the n elements of tensor number `tensor` in the list."""
    low = np.uint64(0xffffffff)
    i = np.arange(n, dtype=np.uint64)
    j = i >> np.uint64(1)
    x, y = j & low, (np.uint64(tensor << 8) ^ (j >> np.uint64(32))) & low
    key = ((seed ^ (seed >> 32)) + step * 0x9E3779B9) & 0xffffffff
    for _ in range(7):
        prod = x * np.uint64(0xD256D193)
        x, y = (prod >> np.uint64(32)) ^ np.uint64(key) ^ y, prod & low
        key = (key + 0x9E3779B9) & 0xffffffff
    return np.where(i & np.uint64(1), y, x)
