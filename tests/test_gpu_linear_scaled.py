"""rra_linear_scaled against the fp64 oracle (needs a GPU).

Bounds as for rra_linear_epilogue's, with S = a_scale w_scale sum_k |a||w|: products of two values in 8 bits are exact in
fp32, each of the K additions is off by at most f = 2^-23 of the running size, the two scales add 3 f / 2 of the product.
"""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from block_util import F, half_step, nan_fill
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu

ACTS = dict(none=rra.ACT_NONE, relu=rra.ACT_RELU, gelu=rra.ACT_GELU, gelu_tanh=rra.ACT_GELU_TANH, silu=rra.ACT_SILU)
E4 = torch.float8_e4m3fn


def _cu(T):
    return torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")


def _run(T, cap, K, N, out, act, bias, residual, seed, in_place=False):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn((cap, K), generator=g) * 60).to(E4)
    w = (torch.randn((N, K), generator=g) * 90).to(E4)
    sa = (0.3 + torch.rand(cap, generator=g)) / 60
    sw = (0.3 + torch.rand(N, generator=g)) / 90 / np.sqrt(K)
    b = torch.randn((N,), generator=g) if bias else None
    r = torch.randn((cap, N), generator=g).to(out) if residual else None
    ad, sad = a.cuda(), sa.cuda()
    nan_fill(ad[T:])                                                # rows past T may hold anything
    nan_fill(sad[T:])
    c = nan_fill(torch.empty((cap, N), dtype=out, device="cuda"))
    rd = r.cuda() if residual else None
    if in_place:
        c.copy_(rd)
        rd = c
    rra.get_device_error(clear=True)
    rra.linear_scaled(ad, sad, w.cuda(), sw.cuda(), _cu(T), 2, c, bias=None if b is None else b.cuda(), act=ACTS[act],
                      residual=rd)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    got = c.cpu()
    a64 = a.float().double().numpy() * sa.double().numpy()[:, None]
    w64 = w.float().double().numpy() * sw.double().numpy()[:, None]
    b64 = b.double().numpy() if bias else None
    r64 = r.double().numpy() if residual else None
    ref = OB.linear_epilogue(a64, w64, b64, act, r64, T)
    x = OB.linear_epilogue(a64, w64, b64, "none", None, T)
    S = np.abs(a64[:T]) @ np.abs(w64).T
    tol = 1.13 * F * ((K + 1.5) * S + (np.abs(b64) if bias else 0.0)) + 16 * F * (1 + np.abs(x))
    if residual:
        tol = tol + F * (np.abs(r64[:T]) + np.abs(ref))
    if out != torch.float32:
        tol = tol + half_step(out) * (np.abs(ref) + tol) + (2.0 ** -25 if out == torch.float16 else 0.0)
    g64 = got.double().numpy()[:T]
    err = np.abs(g64 - ref)
    bad = ~((err <= tol) | (np.isnan(ref) & np.isnan(g64)))         # an input past 464 is NaN in 8 bits, and so are its outputs
    assert not bad.any(), f"{int(bad.sum())} off, worst {np.nanmax(err):.3e}, first {np.argwhere(bad)[0]}"
    if in_place:
        assert torch.equal(got[T:], r[T:])
    else:
        assert bool(torch.isnan(got[T:].float()).all()), "rows past T were written"


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("K,N", [(16, 8), (80, 136), (128, 128), (384, 1152), (1008, 520)])
def test_linear_scaled_sizes(T, K, N):
    _run(T, 320, K, N, torch.float32, "gelu", True, True, seed=T * 31 + K + N)


@pytest.mark.parametrize("cap", [1, 3, 8, 16, 24, 32, 48, 64, 129, 200, 256, 257])
@pytest.mark.parametrize("K,N", [(16, 8), (80, 24), (768, 384), (4096, 512), (1040, 1000)])
def test_linear_scaled_few_rows(cap, K, N):
    for T in {1, cap // 2, cap} - {0}:
        _run(T, cap, K, N, torch.bfloat16, "silu", True, True, seed=T * 31 + K + N)


@pytest.mark.parametrize("cap", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("K,N", [(16, 5000), (80, 8200), (768, 16392), (2512, 9736), (8192, 5128)])
def test_linear_scaled_few_rows_many_columns(cap, K, N):
    """A CTA goes on from columns to columns (where the rows fit its shared memory)."""
    for T in {1, cap}:
        _run(T, cap, K, N, torch.bfloat16, "gelu", True, True, seed=T * 31 + K + N)


@pytest.mark.parametrize("cap,T", [(5, 5), (200, 190), (600, 590)])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
def test_linear_scaled_types(cap, T, act, out):
    for bias, residual in ((False, False), (True, False), (False, True), (True, True)):
        _run(T, cap, 144, 264, out, act, bias, residual, seed=7)
    _run(T, cap, 144, 264, out, act, True, True, seed=8, in_place=True)


@pytest.mark.parametrize("T,cap", [(1, 1), (2, 8), (9, 9), (49, 64), (100, 129), (250, 256)])
@pytest.mark.parametrize("K,N", [(144, 19464), (1040, 13000), (2064, 20488)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
def test_linear_scaled_many_columns(T, cap, K, N, out):
    """Tiles of one CTA, in one round and in several."""
    _run(T, cap, K, N, out, "silu", True, True, seed=T + K, in_place=T % 2 == 1)
    _run(T, cap, K, N, out, "none", False, False, seed=T + K + 1)


@pytest.mark.parametrize("T,cap,K,N", [(4, 4, 4096, 4096), (129, 600, 8192, 264), (40, 64, 1040, 20488), (13, 16, 4096, 8200), (9, 9, 1040, 30008), (61, 64, 2064, 40008), (2569, 2600, 768, 2304),
                                       (300, 300, 80, 8200), (7, 8, 4096, 16384), (16, 16, 2064, 19464), (700, 1200, 1552, 4104), (200, 256, 8208, 1032),
                                       (161, 200, 4112, 4104), (392, 392, 7440, 72), (2, 281, 4784, 136),
                                       (513, 513, 2064, 520), (11000, 11008, 80, 264), (7000, 7000, 144, 1000)])
def test_linear_scaled_exact_integers(T, cap, K, N):
    """Small whole numbers and scales that are powers of two: every product and sum is exact, so the output is too."""
    g = torch.Generator(device="cuda").manual_seed(T + K)
    a = torch.randint(-3, 4, (cap, K), generator=g, device="cuda").float().to(E4)
    w = torch.randint(-3, 4, (N, K), generator=g, device="cuda").float().to(E4)
    sa = 2.0 ** torch.randint(-2, 3, (cap,), generator=g, device="cuda").float()
    sw = 2.0 ** torch.randint(-2, 3, (N,), generator=g, device="cuda").float()
    b = torch.randint(-9, 10, (N,), generator=g, device="cuda").float()
    r = torch.randint(-9, 10, (cap, N), generator=g, device="cuda").float()
    c = torch.full((cap, N), float("nan"), device="cuda")
    rra.linear_scaled(a, sa, w, sw, _cu(T), 2, c, bias=b, residual=r, act=rra.ACT_RELU)
    torch.cuda.synchronize()
    x = (a[:T].double() @ w.double().t()) * sa[:T, None].double() * sw.double()
    assert torch.equal(c[:T].double(), torch.relu(x + b.double()) + r[:T].double())
    assert bool(torch.isnan(c[T:]).all())


@pytest.mark.parametrize("cap", [4, 100, 700])
def test_linear_scaled_every_value(cap):
    """Each of the 254 finite values of the type, times one: it comes back as it is; NaN makes its row's outputs NaN."""
    every = torch.arange(256, dtype=torch.uint8, device="cuda").view(E4)
    keep = torch.isfinite(every.float())
    w = torch.zeros((256, 256), device="cuda")
    w[:, 0] = torch.where(keep, every.float(), torch.zeros_like(every.float()))
    a = torch.zeros((cap, 256), device="cuda")
    a[:, 0] = 1.0
    a[2, 5] = float("nan")
    c = torch.empty((cap, 256), device="cuda")
    ones = torch.ones(max(cap, 256), device="cuda")
    rra.linear_scaled(a.to(E4), ones[:cap], w.to(E4), ones[:256], torch.tensor([0, cap], dtype=torch.int32, device="cuda"), 1, c)
    want = w[:, 0].expand(cap, 256).clone()
    assert torch.equal(c[:2], want[:2]) and torch.equal(c[3:], want[3:]) and bool(torch.isnan(c[2]).all())


@pytest.mark.parametrize("cap", [7, 50, 600])
def test_linear_scaled_scales_of_a_slice(cap):
    """Rows from the middle of a longer buffer: their scales start where they start."""
    g = torch.Generator(device="cuda").manual_seed(cap)
    a = (torch.randn((cap + 5, 128), generator=g, device="cuda") * 60).to(E4)
    w = (torch.randn((72, 128), generator=g, device="cuda") * 60).to(E4)
    sa, sw = torch.rand(cap + 5, generator=g, device="cuda"), torch.rand(72, generator=g, device="cuda")
    whole, part = torch.empty((cap + 5, 72), device="cuda"), torch.empty((cap, 72), device="cuda")
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    rra.linear_scaled(a, sa, w, sw, cu(cap + 5), 1, whole)
    rra.linear_scaled(a[3:cap + 3], sa[3:cap + 3], w, sw, cu(cap), 1, part)
    # (the two calls may take different kernels: sums of 128 products within 128 x 2^-23 of their size, and the scales)
    size = (a[3:cap + 3].float().abs() @ w.float().abs().t()) * sa[3:cap + 3, None] * sw
    assert bool(((whole[3:cap + 3] - part).abs() <= 2 * 131 * F * size).all())


@pytest.mark.parametrize("cap", [8, 100, 400])
def test_linear_scaled_empty_and_bad_count(cap):
    for N, (T, want) in itertools.product((128, 8192), ((0, 0), (cap + 1, rra.DEVERR_INDEX_RANGE), (-1, rra.DEVERR_INDEX_RANGE))):
        a, w = torch.zeros((cap, 64), device="cuda").to(E4), torch.zeros((N, 64), device="cuda").to(E4)
        sa, sw = torch.ones(cap, device="cuda"), torch.ones(N, device="cuda")
        c = torch.full((cap, N), float("nan"), device="cuda")
        rra.get_device_error(clear=True)
        rra.linear_scaled(a, sa, w, sw, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 1, c)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == want
        assert bool(torch.isnan(c).all())


@pytest.mark.parametrize("cap,K,N", [(4, 65536, 64), (2, 16384, 5000), (100, 16384, 9856), (64, 65536, 264), (24, 16384, 24584), (200, 16384, 9728),
                                     (257, 65536, 520), (1500, 16384, 1032)])
def test_long_sums_of_fp32_outputs(cap, K, N):
    """Positive inputs, so that every truncation goes the same way.  A product of the tensor core over 32 elements truncates
    the running sum once, by at most f of it; within a part of K = 1024 the running sums are S_part j / 32, j = 1 .. 32 (10 %
    for the spread): 1.1 x 16.5 f S in all.  The n = K / 1024 parts are added in fp32: 1.1 (n + 1) / 4 f S.  Joining up to 8
    shares adds 4 f S, the scales 1.5 f S, and 1 f S is left for the last addition."""
    g = torch.Generator(device="cuda").manual_seed(cap + K + N)
    a = (0.75 + 0.5 * torch.rand((cap, K), generator=g, device="cuda")).to(E4)
    w = (0.75 + 0.5 * torch.rand((N, K), generator=g, device="cuda")).to(E4)
    sa, sw = 0.5 + torch.rand(cap, generator=g, device="cuda"), 0.5 + torch.rand(N, generator=g, device="cuda")
    c = torch.full((cap, N), float("nan"), device="cuda")
    rra.linear_scaled(a, sa, w, sw, torch.tensor([0, cap], dtype=torch.int32, device="cuda"), 1, c)
    want = torch.empty((cap, N), dtype=torch.float64, device="cuda")
    for n in range(0, N, 1024):
        want[:, n:n + 1024] = a.double() @ w[n:n + 1024].double().t()
    want *= sa.double()[:, None] * sw.double()
    bound = F * (1.1 * 16.5 + 1.1 * (K / 1024 + 1) / 4 + 6.5)
    off = ((c.double() - want).abs() / want).max().item()
    assert off <= bound, f"{off / F:.1f} steps of 2^-23 off, bound {bound / F:.1f}"
