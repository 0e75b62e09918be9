"""rra_qk_norm_rope against the fp64 oracle (needs a GPU).

Bounds, with f = 2^-24: the mean square of d terms, its root, reciprocal and
the products with it and the weight: within (d + 16) f of the value; the angle
is reduced to within 2^-23 of a turn, 2 pi 2^-23 radians, which moves a pair by
that share of its length; products and sums of the rotation: 8 f of the pair's
length; one rounding to the type.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import half_step, nan_fill
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu
f24 = 2.0 ** -24


def _check(got, x, pos, weight, eps, inv_freq, interleaved, rs, dtype):
    d = x.shape[-1]
    ref = OB.norm_rope(x, pos, weight, eps, inv_freq, interleaved, rs)
    y = np.abs(OB.norm_rope(x, None, weight, eps, None, interleaved, 1.0))
    size = y.copy()
    if inv_freq is not None:
        h = len(inv_freq)
        a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
        size[..., a] = size[..., b] = rs * np.hypot(y[..., a], y[..., b])
    tol = size * (d + 16 + 16 + 2 * 2 * np.pi) * f24
    tol += half_step(dtype) * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    err = np.abs(got.double().numpy() - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, worst {np.nanmax(err):.3e}, first {np.argwhere(bad)[0]}"


def _inputs(T, cap, Hq, Hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((cap, Hq + 2 * Hkv, d), generator=g) * 1.7).to(dtype)
    dev = qkv.cuda()
    nan_fill(dev[T:])
    return qkv, dev


@pytest.mark.parametrize("T,cap", [(1, 1), (3, 3), (130, 140)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 7), (8, 2), (32, 8)])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_norm_rope_layouts(T, cap, Hq, Hkv, d, rot, interleaved):
    for dtype, norm in ((torch.bfloat16, True), (torch.float16, False)):
        qkv, dev = _inputs(T, cap, Hq, Hkv, d, dtype, seed=T + Hq + d + rot)
        g = torch.Generator().manual_seed(5)
        pos = torch.randint(0, 1 << 24, (cap,), generator=g, dtype=torch.int32)
        pos[0] = (1 << 24) - 1
        f = (10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))).float() if rot else None
        qw, kw = (1 + 0.2 * torch.randn((2, d), generator=g)) if norm else (None, None)
        q_out = nan_fill(torch.empty((cap, Hq, d), dtype=dtype, device="cuda"))
        k_out = nan_fill(torch.empty((cap, Hkv, d), dtype=dtype, device="cuda"))
        rra.get_device_error(clear=True)
        cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
        rra.qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], pos.cuda() if rot else None, cu, 2, q_out, k_out,
                         f.cuda() if rot else None, q_weight=None if qw is None else qw.cuda(),
                         k_weight=None if kw is None else kw.cuda(), interleaved=interleaved, rope_scale=1.25)
        torch.cuda.synchronize()
        assert rra.get_device_error() == 0
        f64 = f.double().numpy() if rot else None
        for out, sl, w in ((q_out, slice(0, Hq), qw), (k_out, slice(Hq, Hq + Hkv), kw)):
            _check(out.cpu()[:T], qkv[:T, sl].double().numpy(), pos[:T].numpy(), None if w is None else w.double().numpy(),
                   1e-6, f64, interleaved, 1.25, dtype)
            assert bool(torch.isnan(out[T:].float()).all()), "rows past T were written"


@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("d", [64, 128])
def test_qk_norm_rope_cache_write(T, d):
    """Keys and values land in their slots; every other row of the cache keeps its bits; a slot of -1 is reported."""
    Hq, Hkv, R, dtype = 6, 3, 100, torch.bfloat16
    qkv, dev = _inputs(T, T, Hq, Hkv, d, dtype, seed=9)
    g = torch.Generator().manual_seed(T)
    rows = torch.randperm(R, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, 9000, (T,), generator=g, dtype=torch.int32)
    f = 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    w = torch.rand(d, generator=g) + 0.5
    kc, vc = (torch.randn((R, Hkv, d), generator=g).to(dtype) for _ in range(2))
    for bad in (False, True):
        rr = rows.clone()
        if bad:
            rr[T - 1] = -1 if T == 1 else R
        kd, vd = kc.cuda(), vc.cuda()
        q_out = torch.empty((T, Hq, d), dtype=dtype, device="cuda")
        rra.get_device_error(clear=True)
        rra.qk_norm_rope(dev[:, :Hq], dev[:, Hq:Hq + Hkv], pos.cuda(), torch.tensor([0, T], dtype=torch.int32).cuda(), 1,
                         q_out, kd, f.cuda(), q_weight=w.cuda(), k_weight=w.cuda(), v=dev[:, Hq + Hkv:], v_out=vd,
                         kv_rows=rr.cuda())
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == (rra.DEVERR_INDEX_RANGE if bad else 0)
        n = T - 1 if bad else T
        hit = rows[:n].long()
        w64, f64 = w.double().numpy(), f.float().double().numpy()
        _check(q_out.cpu(), qkv[:, :Hq].double().numpy(), pos.numpy(), w64, 1e-6, f64, False, 1.0, dtype)
        if n:
            _check(kd.cpu()[hit], qkv[:n, Hq:Hq + Hkv].double().numpy(), pos[:n].numpy(), w64, 1e-6, f64, False, 1.0, dtype)
        assert torch.equal(vd.cpu()[hit], qkv[:n, Hq + Hkv:])
        rest = torch.ones(R, dtype=torch.bool)
        rest[hit] = False
        assert torch.equal(kd.cpu()[rest], kc[rest]) and torch.equal(vd.cpu()[rest], vc[rest])


def test_qk_norm_rope_in_place_and_slices():
    """In place on the fused buffer, bit for bit what the separate outputs hold; the values stay."""
    T, Hq, Hkv, d = 77, 4, 2, 128
    _, dev = _inputs(T, T, Hq, Hkv, d, torch.float16, seed=3)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).cuda()
    w = torch.ones(d, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty((T, Hq, d), dtype=torch.float16, device="cuda"), torch.empty((T, Hkv, d), dtype=torch.float16,
                                                                                       device="cuda")
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    keep = v.clone()
    rra.qk_norm_rope(q, k, pos, cu, 1, qo, ko, f, q_weight=w, k_weight=w)
    rra.qk_norm_rope(q, k, pos, cu, 1, q, k, f, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, keep)


def test_qk_norm_rope_zero_rows_and_bad_positions():
    T, d = 5, 64
    x = torch.zeros((T, 2, d), dtype=torch.bfloat16, device="cuda")
    x[1:] = 1.0
    f = torch.ones(32, device="cuda")
    w = torch.ones(d, device="cuda")
    pos = torch.tensor([3, 0, -1, 1 << 24, 7], dtype=torch.int32, device="cuda")
    qo, ko = (nan_fill(torch.empty_like(x)) for _ in range(2))
    rra.get_device_error(clear=True)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    rra.qk_norm_rope(x, x.clone(), pos, cu, 1, qo, ko, f, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    assert rra.get_device_error(clear=True) == rra.DEVERR_INDEX_RANGE
    assert bool((qo[0] == 0).all()) and bool((qo[1].float() - 1).abs().max() < 1e-2)     # a row of zeros stays zero
    assert bool(torch.isnan(qo[2:4].float()).all()) and bool(torch.isnan(ko[2:4].float()).all())
    assert bool(torch.isfinite(qo[4].float()).all())
    for T_bad in (-1, T + 1):
        nan_fill(qo)
        rra.qk_norm_rope(x, x.clone(), None, torch.tensor([0, T_bad], dtype=torch.int32, device="cuda"), 1, qo, ko)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == rra.DEVERR_INDEX_RANGE and bool(torch.isnan(qo.float()).all())


def test_qk_norm_rope_rows_past_32_bits():
    """Rows whose offsets pass 2^32 elements, in the input and in the cache."""
    T, Hkv, d, stride = 3, 1, 128, 1 << 31
    big = torch.empty((T - 1) * stride + 3 * d, dtype=torch.bfloat16, device="cuda")
    qkv = big.as_strided((T, 3, d), (stride, d, 1))
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, 3, d), generator=g).to(torch.bfloat16)
    qkv.copy_(x)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    f = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).cuda()
    R = (1 << 25) + 8                                                # 2^32 elements and some
    cache = torch.empty((R, Hkv, d), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([R - 1, 0, R - 3], dtype=torch.int32, device="cuda")
    qo = torch.empty((T, 1, d), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(cache)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    rra.qk_norm_rope(qkv[:, :1], qkv[:, 1:2], pos, cu, 1, qo, cache, f, v=qkv[:, 2:], v_out=vo, kv_rows=rows)
    torch.cuda.synchronize()
    f64 = f.cpu().double().numpy()
    _check(qo.cpu(), x[:, :1].double().numpy(), pos.cpu().numpy(), None, 0.0, f64, False, 1.0, torch.bfloat16)
    _check(cache[rows.long()].cpu(), x[:, 1:2].double().numpy(), pos.cpu().numpy(), None, 0.0, f64, False, 1.0,
           torch.bfloat16)
    assert torch.equal(vo[rows.long()].cpu(), x[:, 2:])
