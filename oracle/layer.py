"""Plain float64 forms of the linear-attention layer's operators (numpy): the token
loop of linear attention with a decay per head and its reverse, the q, k norm with
the rotation, and the gated norm, each with its gradients written out.  Test
infrastructure only; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def la_fwd(q, k, v, log_decay, s0=None):
    """S_t = gamma S_{t-1} + v_t k_t^T, o_t = S_t q_t.  q, k [B,T,H,K], v [B,T,H,V].
    Returns (o, final state, states) with states[t] the state behind token t - 1."""
    B, T, H, K = q.shape
    V = v.shape[-1]
    gamma = np.exp(np.asarray(log_decay, dtype=np.float64))[None, :, None, None]
    S = np.zeros((B, H, V, K)) if s0 is None else np.array(s0, dtype=np.float64)
    o = np.zeros((B, T, H, V))
    states = [S]
    for t in range(T):
        S = gamma * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        o[:, t] = np.einsum("bhvk,bhk->bhv", S, q[:, t])
        states.append(S)
    return o, S, states


def la_bwd(q, k, v, log_decay, s0, d_o, d_final=None):
    """The chain rule through la_fwd in reverse.  Returns (dq, dk, dv, d_s0)."""
    B, T, H, K = q.shape
    gamma = np.exp(np.asarray(log_decay, dtype=np.float64))[None, :, None, None]
    _, _, states = la_fwd(q, k, v, log_decay, s0)
    dS = np.zeros_like(states[0]) if d_final is None else np.array(d_final, dtype=np.float64)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for t in range(T - 1, -1, -1):
        dq[:, t] = np.einsum("bhvk,bhv->bhk", states[t + 1], d_o[:, t])
        dS = dS + d_o[:, t, :, :, None] * q[:, t, :, None, :]
        dk[:, t] = np.einsum("bhvk,bhv->bhk", dS, v[:, t])
        dv[:, t] = np.einsum("bhvk,bhk->bhv", dS, k[:, t])
        dS = gamma * dS
    return dq, dk, dv, dS


def _pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(x, cos, sin, interleaved, sign=1.0):
    """x [B,T,H,D]; cos, sin [B,T,R/2]."""
    y = np.array(x, dtype=np.float64)
    a, b = _pairs(2 * cos.shape[-1], interleaved)
    c, s = cos[:, :, None], sign * sin[:, :, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _inv_rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def norm_rope_fwd(x, w, cos, sin, eps, interleaved):
    """One side (queries or keys): the normed, weighted rows, rotated."""
    return rotate(x * _inv_rms(x, eps) * w, cos, sin, interleaved)


def norm_rope_bwd(x, w, cos, sin, eps, interleaved, dy):
    """Returns (dx, dw)."""
    dn = rotate(dy, cos, sin, interleaved, -1.0)
    r = _inv_rms(x, eps)
    xh, t = x * r, dn * w
    return r * (t - xh * (t * xh).mean(-1, keepdims=True)), (dn * xh).sum((0, 1, 2))


def gated_norm_fwd(x, z, w, eps):
    return x * _inv_rms(x, eps) * w * z / (1.0 + np.exp(-z))


def gated_norm_bwd(x, z, w, eps, dy):
    """Returns (dx, dz, dw)."""
    sg = 1.0 / (1.0 + np.exp(-z))
    act = z * sg
    r = _inv_rms(x, eps)
    xh, t = x * r, dy * act * w
    dx = r * (t - xh * (t * xh).mean(-1, keepdims=True))
    return dx, dy * xh * w * (sg + act * (1.0 - sg)), (dy * act * xh).sum((0, 1, 2))
