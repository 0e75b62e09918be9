"""rra_linear_epilogue against the fp64 oracle (needs a GPU).

Bounds: the product's K terms are exact in fp32 and each addition is off by at
most f = 2^-23 of the running size, so the sum is off by at most K f S,
S = sum_k |a||w|; bias and residual add f each of their sizes; every activation
has a slope of at most 1.13 and is evaluated within 16 f (1 + |x|); the one
rounding to a 16-bit output adds half a step of the result (2^-25 in fp16
below its normal range).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import F, half_step, nan_fill
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu

ACTS = dict(none=rra.ACT_NONE, relu=rra.ACT_RELU, gelu=rra.ACT_GELU, gelu_tanh=rra.ACT_GELU_TANH, silu=rra.ACT_SILU)


def _cu(T):
    return torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")


def _run(T, cap, K, N, dtype, out, act, bias, residual, seed, in_place=False):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn((cap, K), generator=g).to(dtype)
    w = (torch.randn((N, K), generator=g) / np.sqrt(K)).to(dtype)
    b = torch.randn((N,), generator=g) if bias else None
    r = torch.randn((cap, N), generator=g).to(out) if residual else None
    ad = a.cuda()
    nan_fill(ad[T:])                                                # rows past T may hold anything
    c = nan_fill(torch.empty((cap, N), dtype=out, device="cuda"))
    rd = r.cuda() if residual else None
    if in_place:
        c.copy_(rd)
        rd = c
    rra.get_device_error(clear=True)
    rra.linear_epilogue(ad, w.cuda(), _cu(T), 2, c, bias=None if b is None else b.cuda(), act=ACTS[act], residual=rd)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    got = c.cpu()
    a64, w64 = a.double().numpy(), w.double().numpy()
    b64 = b.double().numpy() if bias else None
    r64 = r.double().numpy() if residual else None
    ref = OB.linear_epilogue(a64, w64, b64, act, r64, T)
    x = OB.linear_epilogue(a64, w64, b64, "none", None, T)
    S = np.abs(a64[:T]) @ np.abs(w64).T
    tol = 1.13 * F * (K * S + (np.abs(b64) if bias else 0.0)) + 16 * F * (1 + np.abs(x))
    if residual:
        tol = tol + F * (np.abs(r64[:T]) + np.abs(ref))
    if out != torch.float32:
        tol = tol + half_step(out) * (np.abs(ref) + tol) + (2.0 ** -25 if out == torch.float16 else 0.0)
    g64 = got.double().numpy()
    err = np.abs(g64[:T] - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, worst {np.nanmax(err):.3e}, first {np.argwhere(bad)[0]}"
    if in_place:
        assert torch.equal(got[T:], r[T:])
    else:
        assert bool(torch.isnan(got[T:].float()).all()), "rows past T were written"


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 33, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("K,N", [(8, 8), (72, 136), (64, 128), (384, 1152), (1000, 520)])
def test_linear_epilogue_sizes(T, K, N):
    _run(T, 320, K, N, torch.bfloat16, torch.float32, "gelu", True, True, seed=T * 31 + K + N)


@pytest.mark.parametrize("cap", [1, 3, 8, 16, 24, 32, 48, 64, 129, 200, 256, 257])
@pytest.mark.parametrize("K,N", [(8, 8), (72, 24), (768, 384), (4096, 512), (1032, 1000)])
def test_linear_epilogue_few_rows(cap, K, N):
    """The serving form: a handful of rows, all in use and not."""
    for T in {1, cap // 2, cap} - {0}:
        _run(T, cap, K, N, torch.bfloat16, torch.bfloat16, "silu", True, True, seed=T * 31 + K + N)


@pytest.mark.parametrize("cap,T", [(5, 5), (200, 190)])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                       (torch.float16, torch.float32), (torch.bfloat16, torch.float16),
                                       (torch.float16, torch.bfloat16)])
def test_linear_epilogue_types(cap, T, act, dtype, out):
    for bias, residual in ((False, False), (True, False), (False, True), (True, True)):
        _run(T, cap, 136, 264, dtype, out, act, bias, residual, seed=7)
    _run(T, cap, 136, 264, dtype, out, act, True, True, seed=8, in_place=True)


@pytest.mark.parametrize("T,cap,K,N", [(4, 4, 4096, 4096), (129, 600, 8192, 264), (2569, 2600, 768, 2304),
                                       (300, 300, 72, 8200), (700, 1200, 1544, 4104), (200, 256, 8200, 1032),
                                       (161, 200, 4104, 4104), (392, 392, 7440, 72), (300, 1000, 4784, 136), (2, 281, 4784, 136),
                                       (513, 513, 2056, 520), (200, 200, 1032, 16392),
                                       # a last round of few tiles, cut in four, in two, and past the last column
                                       (11000, 11000, 72, 512), (11000, 11008, 72, 264), (11000, 11000, 584, 264),
                                       (7000, 7000, 136, 1000)])
def test_linear_epilogue_exact_integers(T, cap, K, N):
    """Small whole numbers: every product and sum is exact, so the output is too."""
    g = torch.Generator(device="cuda").manual_seed(T + K)
    a = torch.randint(-3, 4, (cap, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-3, 4, (N, K), generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randint(-9, 10, (N,), generator=g, device="cuda").float()
    r = torch.randint(-9, 10, (cap, N), generator=g, device="cuda").float()
    c = torch.full((cap, N), float("nan"), device="cuda")
    rra.linear_epilogue(a, w, _cu(T), 2, c, bias=b, residual=r, act=rra.ACT_RELU)
    torch.cuda.synchronize()
    want = torch.relu(a[:T].double() @ w.double().t() + b.double()) + r[:T].double()
    assert torch.equal(c[:T].double(), want)
    assert bool(torch.isnan(c[T:]).all())


def test_linear_epilogue_special_values():
    """NaN and infinities go where the formula sends them, and nowhere else."""
    for cap in (4, 130):
        a = torch.ones((cap, 64), dtype=torch.bfloat16, device="cuda")
        a[1, 3], a[2, 5], a[3, 6] = float("nan"), float("inf"), -float("inf")
        w = torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
        c = torch.empty((cap, 16), dtype=torch.float32, device="cuda")
        for act, want in (("none", (64.0, "nan", np.inf, -np.inf)), ("relu", (64.0, "nan", np.inf, 0.0)),
                          ("gelu", (64.0, "nan", np.inf, None)), ("silu", (64.0, "nan", np.inf, None))):
            rra.linear_epilogue(a, w, torch.tensor([0, cap], dtype=torch.int32, device="cuda"), 1, c, act=ACTS[act])
            got = c.cpu().numpy()
            for i, x in enumerate(want):
                if x == "nan":
                    assert np.isnan(got[i]).all()
                elif x is not None:
                    assert np.all(got[i] == x), (act, i, got[i])
            assert np.all(got[4:] == 64.0)


def test_linear_epilogue_empty_and_bad_count():
    for cap in (8, 256):
        a, w = torch.zeros((cap, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((128, 64), dtype=torch.bfloat16,
                                                                                         device="cuda")
        for T, want in ((0, 0), (cap + 1, rra.DEVERR_INDEX_RANGE), (-1, rra.DEVERR_INDEX_RANGE)):
            c = torch.full((cap, 128), float("nan"), device="cuda")
            rra.get_device_error(clear=True)
            rra.linear_epilogue(a, w, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 1, c)
            torch.cuda.synchronize()
            assert rra.get_device_error(clear=True) == want
            assert bool(torch.isnan(c).all())
