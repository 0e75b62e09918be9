"""Shared by the tests of the block operators: inputs, and the bound on a
computed attention row.

Attention.  With u the half step of the 16-bit type (finfo.eps / 2) and
f = 2^-23 (an fp32 operation of the tensor cores, which may truncate), for a row of m keys:
each score is a sum of d products, off by at most ds = d f scale sum|q||k|
(relative to the weights: a factor exp(+-ds)), base-2 exponentials add 4 f
plus f per unit of the exponent (at most 160 units count: smaller weights are
below 2^-149); each weight enters the product rounded (u); the sums over m keys
add m f each for the product and the normaliser.  So |o - ref| <=
mag (u + 2 ds + m 2 f + 200 f) + u |o|, mag = sum_j p_j |v_j|.  In fp16 a weight
below the type's normal range is rounded to a fixed step instead: the weights carry a
factor 2^7 against a largest weight of at least 1, so the error is at most 2^-25 / 2^7 of
the sum of weights for each key, 2^-32 sum_j |v_j| in all.
"""
import numpy as np
import torch

from oracle import block as OB

F = 2.0 ** -23


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def attention_bound(q, k, v, scale, last, o, mag, dtype):
    q, k = np.abs(np.asarray(q, np.float64)), np.abs(np.asarray(k, np.float64))
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    u = half_step(dtype)
    tol = np.zeros(o.shape)
    for h in range(Hq):
        for i in range(n):
            m = int(last[i]) + 1
            if m <= 0:
                continue
            ds = d * F * scale * float((k[:m, h // G] @ q[i, h]).max())
            tol[i, h] = mag[i, h] * (u + 2 * ds + 2 * m * F + 200 * F) + u * np.abs(o[i, h])
            if dtype == torch.float16:
                tol[i, h] += 2.0 ** -32 * np.abs(v[:m, h // G]).sum(0)
    # fp16 results below the normal range are rounded to a fixed step.
    return tol + (2.0 ** -24 if dtype == torch.float16 else 0.0)


def check_rows(got, q, k, v, scale, last, dtype, rows=None):
    """got [n, Hq, d] (cpu tensor) against the oracle, at `rows` only when given."""
    q, k, v = (x.double().numpy() for x in (q, k, v))
    got = got.double().numpy()
    last = np.asarray(last)
    if rows is not None:
        q, got, last = q[rows], got[rows], last[rows]
    o, mag = OB.attend_rows(q, k, v, scale, last)
    tol = attention_bound(q, k, v, scale, last, o, mag, dtype)
    err = np.abs(got - o)
    assert np.all(np.isfinite(got)), "not finite"
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} elements off, worst {err[bad].max():.3e} (bound {tol[bad].min():.3e}) " \
                          f"first at {np.argwhere(bad)[0]}"


def nan_fill(t):
    t.view(torch.uint8).fill_(0xFF)
    return t
