"""CPU oracle (fp64 numpy) of a language model's block on packed rows: the
linear layer with its epilogue, the per-head norms with the position rotation,
and attention of rows over the keys each of them sees.  Plain definitions,
sharing no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def activate(x, act):
    x = np.asarray(x, dtype=np.float64)
    if act == "relu":
        return np.maximum(x, 0.0)
    if act == "gelu":
        return 0.5 * x * (1.0 + _erf(x / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    if act == "silu":
        return x / (1.0 + np.exp(-x))
    return x


def linear_epilogue(a, w, bias, act, residual, T):
    """[T, N]: act(a w^T + bias) + residual for the rows t < T."""
    x = np.asarray(a, dtype=np.float64)[:T] @ np.asarray(w, dtype=np.float64).T
    if bias is not None:
        x = x + np.asarray(bias, dtype=np.float64)[None, :]
    x = activate(x, act)
    if residual is not None:
        x = x + np.asarray(residual, dtype=np.float64)[:T]
    return x


def norm_rope(x, positions, weight, eps, inv_freq, interleaved, rope_scale):
    """x [T, H, d]: RMS norm per head row (weight not None), then the rotation (inv_freq not None)."""
    x = np.asarray(x, dtype=np.float64)
    T, H, d = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / d + eps) * np.asarray(weight, dtype=np.float64)
    y = x.copy()
    if inv_freq is None:
        return y
    half = len(inv_freq)
    for t in range(T):
        for i in range(half):
            ang = float(positions[t]) * float(inv_freq[i])
            c, s = rope_scale * math.cos(ang), rope_scale * math.sin(ang)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return y


def attend_rows(q, k, v, scale, last):
    """q [n, Hq, d] over k, v [m, Hkv, d]: row i sees the keys j <= last[i].

    Returns (o, mag): the attention output, zero for a row that sees nothing,
    and mag = sum_j p_j |v_j|, the size against which rounding is counted."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(Hq):
        for i in range(n):
            m = int(last[i]) + 1
            if m <= 0:
                continue
            s = scale * (k[:m, h // G] @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ v[:m, h // G]
            mag[i, h] = p @ np.abs(v[:m, h // G])
    return o, mag


def to_e4m3(v):
    """Each v rounded to the nearest value in 8 bits (e4m3: normal from 2^-6, steps of 2^-9 below, up to 448), ties to even."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def rms_norm(x, residual, weight, eps):
    """(sum, y): x + residual (or x), and its RMS norm by rows, times weight."""
    r = np.asarray(x, dtype=np.float64)
    if residual is not None:
        r = r + np.asarray(residual, dtype=np.float64)
    y = r / np.sqrt((r * r).sum(-1, keepdims=True) / r.shape[-1] + eps)
    return r, y if weight is None else y * np.asarray(weight, dtype=np.float64)


def row_scale(y):
    """The scale of each row in 8 bits."""
    return np.maximum(np.abs(y).max(-1) / 448.0, 2.0 ** -100)


def cached_rows(pages, table, n):
    """The first n rows of a sequence whose pages [num_pages, page, ...] its row of the table lists."""
    page = pages.shape[1]
    return np.stack([pages[int(table[j // page]), j % page] for j in range(n)]) if n else pages[0, :0]
