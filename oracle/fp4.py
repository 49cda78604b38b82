"""Oracle of the four-bit token operators, in float64 (NumPy), from the format's
definition: groups of 32 values with one scale byte s, codes of a sign and a size
of 0, 0.5, 1, 1.5, 2, 3, 4 or 6, value = code * 2^(s - 127), NaN where s = 255.
"""
from __future__ import annotations

import math

import numpy as np

SIZES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def values(codes, scales):
    """codes [..., n/2], scales [..., n/32] uint8 -> values [..., n]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    nib = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.int64)
    nib[..., 0::2], nib[..., 1::2] = codes & 15, codes >> 4
    v = np.where(nib & 8, -1.0, 1.0) * SIZES[nib & 7]
    unit = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(scales.shape + (32,)) * unit[..., None]).reshape(v.shape)


def quantise(x):
    """x [..., n] -> (codes [..., n/2], scales [..., n/32]) uint8: the code of
    each value is searched among all of them."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    flat = g.reshape(-1, 32)
    nib = np.zeros(flat.shape, np.int64)
    scales = np.zeros(len(flat), np.uint8)
    for i, group in enumerate(flat):
        if not np.all(np.isfinite(group)):
            scales[i] = 255
            continue
        a = np.abs(group).max()
        e = -125
        while e < 125 and a >= math.ldexp(7.0, e):
            e += 1
        scales[i] = e + 127
        r = np.abs(group) / math.ldexp(1.0, e)
        d = np.abs(r[:, None] - SIZES)
        best = d.min(1, keepdims=True)
        even = np.where(d == best, np.where(np.arange(8) % 2 == 0, 0, 1), 2)  # the even one of a tie
        nib[i] = np.argmin(even, 1) | (np.signbit(group).astype(np.int64) << 3)
    nib = nib.reshape(x.shape)
    return (nib[..., 0::2] | nib[..., 1::2] << 4).astype(np.uint8), scales.reshape(g.shape[:-1])


def place(table, pages, page, b, i):
    """(page, row) of place i of sequence b, None without one."""
    if i < 0 or i >= table.shape[1] * page:
        return None
    p = int(table[b, i // page])
    return (p, i % page) if 0 <= p < pages else None


def append(k, v, codes, scales, table, start=None, count=None):
    """k, v [B,T,Hk,D] into copies of the cache's arrays."""
    codes, scales = np.array(codes), np.array(scales)
    B, T = k.shape[:2]
    for b in range(B):
        n = T if count is None else min(max(int(count[b]), 0), T)
        for t in range(n):
            at = place(table, codes.shape[0], codes.shape[3], b, (0 if start is None else int(start[b])) + t)
            if at is not None:
                for i, x in enumerate((k, v)):
                    codes[at[0], i, :, at[1]], scales[at[0], i, :, at[1]] = quantise(x[b, t])
    return codes, scales


def read(codes, scales, table, T, start=None, count=None):
    """-> k, v [B,T,Hk,D]: zeros without a place and past count."""
    B, (pages, _, Hk, page, half) = len(table), codes.shape
    out = np.zeros((2, B, T, Hk, 2 * half))
    for b in range(B):
        n = T if count is None else min(max(int(count[b]), 0), T)
        for t in range(n):
            at = place(table, pages, page, b, (0 if start is None else int(start[b])) + t)
            if at is not None:
                out[:, b, t] = values(codes[at[0], :, :, at[1]], scales[at[0], :, :, at[1]])
    return out[0], out[1]


def attention(q, codes, scales, table, length=None, q_len=None, causal=False, scale=None):
    """q [B,Tq,Hq,D] -> (out, the weighted mean of |v|, the largest scaled sum
    |q k|); rows past q_len and rows without keys are zero."""
    B, Tq, Hq, D = q.shape
    pages, _, Hk, page, _ = codes.shape
    cap = table.shape[1] * page
    scale = D ** -0.5 if scale is None else scale
    out, mean_abs, worst = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for b in range(B):
        n = cap if length is None else min(max(int(length[b]), 0), cap)
        t_n = Tq if q_len is None else min(max(int(q_len[b]), 0), Tq)
        if n == 0:
            continue
        ids = table[b, :(n + page - 1) // page].astype(np.int64)
        there = np.repeat((ids >= 0) & (ids < pages), page)[:n]
        ids = np.where((ids >= 0) & (ids < pages), ids, 0)
        # [columns, 2, Hk, page, D] -> [2, Hk, tokens, D]
        kv = values(codes[ids], scales[ids]).transpose(1, 2, 0, 3, 4).reshape(2, Hk, -1, D)[:, :, :n]
        for i in range(t_n):
            see = there.copy()
            if causal:
                see &= np.arange(n) <= n - t_n + i
            if not see.any():
                continue
            for h in range(Hq):
                k, v = kv[0, h // (Hq // Hk)][see], kv[1, h // (Hq // Hk)][see]
                x = q[b, i, h].astype(np.float64)
                s = (k @ x) * scale
                worst = max(worst, float((np.abs(k) @ np.abs(x)).max()) * scale)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, i, h], mean_abs[b, i, h] = p @ v, p @ np.abs(v)
    return out, mean_abs, worst
