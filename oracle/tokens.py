"""Oracle of the token operators, in float64 (NumPy), from their formulas:
matrix product with bias, activation and residual; head norm and rotary
positions with several axes; attention over a shared prefix and own keys.

Beside its results each function gives the sums of absolute values that
bound what rounding can do to them.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if act == "quick_gelu":
        return z / (1.0 + np.exp(-1.702 * z))
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    assert act == "none"
    return z


def linear(x, w, bias=None, residual=None, act="none"):
    """x [M,K], w [N,K] -> (out [M,N], sum_k |x w| + |bias|, |residual|)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    z = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
        size = size + np.abs(bias)
    y = activation(z, act)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, size


def rope(x, pos, freqs, weight=None, eps=1e-6, interleaved=False):
    """x [B,T,H,D], pos [B,T,A], freqs [A,half] -> (y, |u_p| + |u_q| of each
    element's pair: its own |u| where it does not rotate)."""
    x = np.asarray(x, np.float64)
    u = x
    if weight is not None:
        u = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = freqs.shape[1]
    phi = np.zeros(pos.shape[:2] + (half,))
    for a in range(freqs.shape[0]):
        phi += pos[..., a:a + 1].astype(np.float64) * freqs[a].astype(np.float64)
    c, s = np.cos(phi)[:, :, None], np.sin(phi)[:, :, None]
    if interleaved:
        i0, i1 = np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)
    else:
        i0, i1 = np.arange(half), np.arange(half, 2 * half)
    y, size = u.copy(), np.abs(u)
    y[..., i0] = u[..., i0] * c - u[..., i1] * s
    y[..., i1] = u[..., i1] * c + u[..., i0] * s
    size[..., i0] = size[..., i1] = np.abs(u[..., i0]) + np.abs(u[..., i1])
    return y, size


def prefix_attention(q, kp, vp, ko, vo, own_len=None, q_len=None, own_mask=None, causal=False,
                     scale=None):
    """q [B,Tq,Hq,D]; kp, vp [P,Hk,D]; ko, vo [B,S,Hk,D] -> (out, the
    weighted mean of |v|, the largest scaled sum |q k|); rows past q_len and
    rows without keys are zero."""
    B, Tq, Hq, D = q.shape
    P, Hk = kp.shape[:2]
    S = ko.shape[1]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros(q.shape)
    mean_abs = np.zeros(q.shape)
    worst = 0.0
    for b in range(B):
        n = S if own_len is None else int(min(max(own_len[b], 0), S))
        t_n = Tq if q_len is None else int(min(max(q_len[b], 0), Tq))
        for i in range(t_n):
            see = np.ones(n, bool)
            if own_mask is not None:
                see &= np.asarray(own_mask[b, :n]) != 0
            if causal:
                see &= np.arange(n) <= n - t_n + i
            for h in range(Hq):
                hk = h // G
                k = np.concatenate([kp[:, hk], ko[b, :n, hk][see]]).astype(np.float64)
                v = np.concatenate([vp[:, hk], vo[b, :n, hk][see]]).astype(np.float64)
                if not len(k):
                    continue
                qv = q[b, i, h].astype(np.float64)
                s = (k @ qv) * scale
                worst = max(worst, float((np.abs(k) @ np.abs(qv)).max()) * scale)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, i, h] = p @ v
                mean_abs[b, i, h] = p @ np.abs(v)
    return out, mean_abs, worst
