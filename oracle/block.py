"""Plain float64 forms of what surrounds the linear-attention layer in its block (numpy):
the residual's addition with the RMS norm and its gradients, 8-bit floats with scales, the
axes of a rotation by several positions, the gradients' norm and clipping, and states in 8
bits.  Test infrastructure only; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

LEAST = 2.0 ** -126  # the least scale


def add_norm_fwd(x, residual, w, eps):
    """Returns (y, h) for rows of the last dimension."""
    h = np.asarray(x, dtype=np.float64) + (0.0 if residual is None else residual)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w, h


def add_norm_bwd(h, w, eps, dy, dh=None):
    """Returns (d, dw): the gradient of h's terms and the weight's."""
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, t = h * r, dy * w
    d = r * (t - n * (t * n).mean(-1, keepdims=True))
    return d + (0.0 if dh is None else dh), (dy * n).reshape(-1, h.shape[-1]).sum(0)


def add_norm_bwd_sizes(h, w, eps, dy, dh=None):
    """The same sums over the sizes of their terms: what rounding errors are relative to."""
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, t = np.abs(h * r), np.abs(dy * w)
    d = r * (t + n * (t * n).mean(-1, keepdims=True))
    return d + (0.0 if dh is None else np.abs(dh)), (np.abs(dy) * n).reshape(-1, h.shape[-1]).sum(0)


def e4m3_numbers():
    """The finite numbers of e4m3 from 0 up: sign, 4 bits of exponent (bias 7), 3 of mantissa;
    the largest code is NaN."""
    sub = [m / 8 * 2.0 ** -6 for m in range(8)]
    return np.array(sub + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def e4m3(x):
    """The nearest of them, ties to the even code; past the largest, the largest."""
    table = e4m3_numbers()
    a = np.minimum(np.abs(x), table[-1])
    i = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo, hi = a - table[i - 1], table[i] - a
    up = (hi < lo) | ((hi == lo) & (i % 2 == 0))
    return np.sign(x) * np.where(up, table[i], table[i - 1])


def quantise(y, group):
    """(values, scales) of rows in groups of columns (0: the whole row)."""
    g = y.reshape(*y.shape[:-1], -1, group or y.shape[-1])
    s = np.maximum(np.abs(g).max(-1, keepdims=True) / 448.0, LEAST)
    return e4m3(g / s).reshape(y.shape), s[..., 0]


def axis_of_pair(sections, alternating):
    """The axis of each pair."""
    n = len(sections)
    if not alternating:
        return np.repeat(np.arange(n), sections)
    pairs = sum(sections)
    return np.array([i % n if i // n < sections[i % n] else 0 for i in range(pairs)], dtype=np.int64)


def angles(cos, sin, positions, sections, alternating):
    """Each token's cosines and sines [B,T,R/2] from the tables and positions [axes,B,T]."""
    axis = axis_of_pair(sections, alternating)
    at = np.moveaxis(positions[axis], 0, -1)
    i = np.arange(len(axis))
    return cos[at, i], sin[at, i]


def clip(grads, max_norm):
    """Returns (norm, clipped)."""
    norm = np.sqrt(sum(float((g * g).sum()) for g in grads))
    by = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return norm, [g * by for g in grads]


def park(states):
    """(codes, scales) of float32 rows; the scales are the float32 products by 1/127, and the
    codes count those."""
    x = np.asarray(states, dtype=np.float64)
    s = np.abs(x).max(-1).astype(np.float32) * (np.float32(1) / np.float32(127))
    s = np.maximum(s.astype(np.float64), LEAST)
    return np.rint(x / s[..., None]), s
