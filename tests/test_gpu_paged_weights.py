"""How exactly rra_attend_paged weighs the values of a few rows (needs a GPU).

One warp's products there are bound by the read of the cache, so a weight enters them as two values of the input's type, the second
what the first's rounding left.  With u the half step of the type and f = 2^-23 (an fp32 operation of the tensor cores, which may
truncate), a weight so is off by u^2 of itself, and for a row of m keys the rest is in fp32: a score is a sum of d products,
then a product with the scale, whose constant is rounded too, off by at most ds = (d + 4) f scale sum|q||k|, which goes into the
weights and into their sum; an exponential adds 4 f and f for each unit of its exponent (160 at most), twice where partial
results are joined, and once more in the sum of the weights: under 500 f; the products' sums take 2 m additions and the weights' m,
under 4 m f with the joins'.  So before its last rounding a result is off by t <= mag (u^2 + 2 ds + (4 m + 500) f),
mag = sum_j p_j |v_j|, and then by u (|o| + t).  In fp16 the second value of a weight is rounded to a fixed step at the
smallest, 2^-25 against weights of at least 2^7 at the largest: 2^-32 sum_j |v_j| more; and a result to one of 2^-25.

With weights rounded to one value the error is up to u mag, in bf16 some tens of t, which results that cancel show.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import F, half_step
from oracle import block as OB
from ragged_attention_token_gb300 import rra
from test_gpu_attend_paged import Paged

pytestmark = pytest.mark.gpu


def _check(p, Hq, Hkv, d, max_new, max_kv):
    assert rra.attend_paged_workspace(len(p.kv), p.cap, max_new, max_kv, Hq, Hkv, d) is None, "not the kernel of a few rows"
    p.call(max_new=max_new, max_kv=max_kv)
    torch.cuda.synchronize()
    got, u, scale, G = p.o.cpu().double().numpy(), half_step(p.dtype), d ** -0.5, Hq // Hkv
    for b, (n, m) in enumerate(zip(p.new, p.kv)):
        if n == 0 or m == 0:
            continue
        s0 = int(p.at[b])
        q, k, v = (x.double().numpy() for x in (p.q[s0:s0 + n, :Hq], p.k[b], p.v[b]))
        last = m - n + np.arange(n)
        o, mag = OB.attend_rows(q, k, v, scale, last)
        for i in range(n):
            keys = int(last[i]) + 1
            for h in range(Hq):
                ds = (d + 4) * F * scale * float((np.abs(k[:keys, h // G]) @ np.abs(q[i, h])).max())
                t = mag[i, h] * (u * u + 2 * ds + (4 * keys + 500) * F)
                if p.dtype is torch.float16:
                    t = t + 2.0 ** -32 * np.abs(v[:keys, h // G]).sum(0)
                tol = t + u * (np.abs(o[i, h]) + t) + (2.0 ** -25 if p.dtype is torch.float16 else 0.0)
                err = np.abs(got[s0 + i, h] - o[i, h])
                assert np.all(err <= tol), f"sequence {b} row {i} head {h}: {(err / tol).max():.2f} times the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv,d", [(12, 12, 64), (8, 2, 128), (7, 1, 64), (16, 1, 128)])
def test_weights_of_next_tokens(Hq, Hkv, d, dtype):
    kv = [1, 2, 3, 4, 5, 8, 15, 16, 17, 39, 64, 100, 197]
    _check(Paged([1] * len(kv), kv, Hq, Hkv, d, 16, dtype, seed=Hq), Hq, Hkv, d, 1, 197)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_a_few_tokens(d, dtype):
    kv = [4, 5, 9, 33, 130]
    _check(Paged([4] * 5, kv, 8, 2, d, 32, dtype, seed=d, joint=True), 8, 2, d, 4, 130)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_joined_across_a_cluster(d, dtype):
    _check(Paged([1, 1], [2048, 1500], 8, 2, d, 64, dtype, seed=d + 1), 8, 2, d, 1, 2048)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_of_large_groups(dtype):
    _check(Paged([2, 1], [30, 9], 129, 1, 64, 16, dtype, seed=3), 129, 1, 64, 2, 30)
