"""rra_rms_norm against the fp64 oracle (needs a GPU).

Bounds, f = 2^-24 (half a step of fp32).  r = x + residual is off by f |r|.  A thread adds up to 32 squares in a row, then 10
more additions join 1024 threads: the sum of squares is within (32 + 10 + 1 + 2) f of itself (2 for r's own error), the mean
and eps add 2 f; the reciprocal root halves that and adds 4 f of its own (2 units), the products with the weight and r 2 f,
r's error 1 f: (47 / 2 + 7) f < 32 f.  So y is within 32 f |y| and one rounding; the scale, a maximum of |y| divided once,
within 33 f; y / scale, by a reciprocal and a product, within (32 + 33 + 2) f = 67 f of itself before its one rounding: a
result lies between the roundings of the exact quotient's two ends.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import half_step, nan_fill
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
BF, FP, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def _cu(T):
    return torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")


def _near(got, want, rel, dtype):
    tol = rel * np.abs(want)
    if dtype is not F32:
        tol = tol + half_step(dtype) * (np.abs(want) + tol) + (2.0 ** -25 if dtype is FP else 2.0 ** -134)
    else:
        tol = tol + 2.0 ** -149
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first {np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}"


def _run(T, cap, N, dtype, out, res, weight, seed, eps=1e-6, gain=1.0, alias=()):
    """res: the residual's type or None; alias: "sum" (into the residual), "sum_x", "y" (into x)."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((cap, N), generator=g) * gain).to(dtype)
    r = None if res is None else (torch.randn((cap, N), generator=g) * gain * 2).to(res)
    w = 1 + 0.3 * torch.randn(N, generator=g) if weight else None
    nan_fill(x[T:])                                                 # rows past T may hold anything
    xd, rd = x.cuda(), None if r is None else r.cuda()
    sd = None if r is None else rd if "sum" in alias else xd if "sum_x" in alias else nan_fill(torch.empty_like(rd))
    yd = xd if "y" in alias else nan_fill(torch.empty((cap, N), dtype=out, device="cuda"))
    sc = nan_fill(torch.empty(cap, device="cuda")) if out is E4 else None
    before = [None if t is None else t[T:].cpu().clone().view(torch.uint8) for t in (yd, sd, sc)]
    rra.get_device_error(clear=True)
    rra.rms_norm(xd, _cu(T), 2, yd, weight=None if w is None else w.cuda(), residual=rd, sum_out=sd, scale=sc, eps=eps)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    for t, b in zip((yd, sd, sc), before):
        assert t is None or torch.equal(t[T:].cpu().view(torch.uint8), b), "rows past T were written"
    s64, y64 = OB.rms_norm(x[:T].double().numpy(), None if r is None else r[:T].double().numpy(),
                           None if w is None else w.double().numpy(), float(np.float32(eps)))
    if r is not None:
        _near(sd[:T].cpu().double().numpy(), s64, F, res)
    got = yd[:T].cpu().double().numpy()
    if out is not E4:
        _near(got, y64, 32 * F, out)
        return
    scale = OB.row_scale(y64)
    _near(sc[:T].cpu().double().numpy(), scale, 33 * F, F32)
    v = y64 / scale[:, None]
    lo, hi = OB.to_e4m3(v - np.abs(v) * 67 * F), OB.to_e4m3(v + np.abs(v) * 67 * F)
    assert np.all((lo <= got) & (got <= hi))


@pytest.mark.parametrize("N", [8, 40, 256, 1016, 1024, 1032, 2048, 2056, 4096, 5120, 8200, 16384, 32768])
@pytest.mark.parametrize("T,cap", [(1, 1), (5, 9), (67, 67)])
def test_rms_norm_sizes(T, cap, N):
    for out, res in ((E4, BF), (BF, F32), (E4, None)):
        _run(T, cap, N, BF, out, res, True, seed=T + N)


@pytest.mark.parametrize("N", [8, 264, 520, 776, 1032, 4096, 4104, 6144, 6152])
def test_rms_norm_many_rows(N):
    """Enough rows that a thread has several, one after the other."""
    for T, out, res in ((1999, E4, BF), (2001, BF, None), (1300, E4, F32)):
        _run(T, 2001, N, BF, out, res, True, seed=N)


@pytest.mark.parametrize("N", [6160, 8192, 8200, 12288, 12296, 16384])
def test_rms_norm_many_long_rows(N):
    for T, cap, out, res in ((701, 720, E4, BF), (330, 330, BF, BF), (640, 1300, BF, None), (500, 500, E4, F32)):
        _run(T, cap, N, BF, out, res, True, seed=T + N)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("res", ["none", "same", "fp32"])
@pytest.mark.parametrize("weight", [False, True])
def test_rms_norm_types(dtype, eight, res, weight):
    for N in (264, 3592):
        _run(23, 31, N, dtype, E4 if eight else dtype, {"none": None, "same": dtype, "fp32": F32}[res], weight, seed=N)


@pytest.mark.parametrize("N", [136, 2304])
def test_rms_norm_in_place(N):
    _run(20, 23, N, BF, E4, BF, True, seed=1, alias=("sum",))
    _run(20, 23, N, BF, E4, BF, True, seed=2, alias=("sum_x",))
    _run(20, 23, N, FP, FP, F32, True, seed=3, alias=("sum", "y"))
    _run(20, 23, N, BF, BF, None, False, seed=4, alias=("y",))


@pytest.mark.parametrize("gain", [1e-12, 3e-3, 3e4])
def test_rms_norm_small_and_large_values(gain):
    """Rows that eps outweighs, and rows of large values."""
    _run(9, 9, 520, BF, E4, BF, True, seed=5, gain=gain)
    _run(9, 9, 520, BF, BF, F32, True, seed=6, gain=gain, eps=0.0)


def test_rms_norm_special_rows():
    """A row of zeros, a NaN, an infinity: each keeps to its row."""
    for N in (64, 4096):
        x = torch.ones((5, N), dtype=BF, device="cuda")
        x[1], x[2, 3], x[3, N - 1] = 0.0, float("nan"), float("inf")
        y, sc = torch.empty((5, N), dtype=E4, device="cuda"), torch.empty(5, device="cuda")
        rra.rms_norm(x, _cu(5), 2, y, scale=sc, eps=0.0 if N == 64 else 1e-6)
        y, sc = y.float().cpu(), sc.cpu()
        assert bool((y[0] == 448).all() and (y[4] == 448).all()) and abs(sc[0].item() * 448 - 1) < 1e-5
        if N == 64:
            assert bool(torch.isnan(y[1]).all() and torch.isnan(sc[1]))     # 0 * rsqrt(0)
        else:
            assert bool((y[1] == 0).all()) and sc[1].item() == 2.0 ** -100
        assert bool(torch.isnan(y[2]).all() and torch.isnan(sc[2]))
        assert bool(torch.isnan(sc[3]) and torch.isnan(y[3]).all())         # the infinity itself becomes inf * 0
        y16 = torch.empty((5, N), dtype=BF, device="cuda")
        rra.rms_norm(x, _cu(5), 2, y16)
        y16 = y16.float().cpu()
        assert bool((y16[0] == 1).all() and (y16[1] == 0).all() and torch.isnan(y16[2]).all())
        assert bool((y16[3, :N - 1] == 0).all() and torch.isnan(y16[3, N - 1]))


@pytest.mark.parametrize("N", [64, 4096])
def test_rms_norm_squares_past_the_range(N):
    """A sum of squares beyond fp32's range: zeros, also where the product with the weight is beyond it, and its row alone."""
    x = torch.ones((3, N), dtype=BF, device="cuda")
    x[1, 5] = 3e38
    for w in (1.0, 2.0):
        weight = torch.full((N,), w, device="cuda")
        y, sc = torch.empty((3, N), dtype=E4, device="cuda"), torch.empty(3, device="cuda")
        rra.rms_norm(x, _cu(3), 2, y, weight=weight, scale=sc)
        y16 = torch.empty((3, N), dtype=BF, device="cuda")
        rra.rms_norm(x, _cu(3), 2, y16, weight=weight)
        assert bool((y.float()[1] == 0).all() and (y16[1] == 0).all()) and sc[1].item() == 2.0 ** -100
        assert bool((y.float()[::2] == 448).all() and (y16[::2] == w).all())


@pytest.mark.parametrize("N", [64, 4096])
def test_rms_norm_empty_and_bad_count(N):
    x = torch.ones((6, N), dtype=BF, device="cuda")
    for T, want in ((0, 0), (7, rra.DEVERR_INDEX_RANGE), (-1, rra.DEVERR_INDEX_RANGE)):
        y = torch.full((6, N), float("nan"), dtype=BF, device="cuda")
        rra.get_device_error(clear=True)
        rra.rms_norm(x, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 1, y)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == want
        assert bool(torch.isnan(y).all())


def test_rms_norm_rows_past_32_bits():
    """A buffer of more than 2^32 elements: its last row."""
    N = 32768
    cap = (1 << 17) + 3
    x = torch.zeros((cap, N), dtype=BF, device="cuda")
    x[cap - 1] = torch.randn(N, device="cuda").to(BF)
    y, sc = torch.empty((cap, N), dtype=E4, device="cuda"), torch.empty(cap, device="cuda")
    rra.rms_norm(x, _cu(cap), 2, y, scale=sc)
    _, y64 = OB.rms_norm(x[cap - 1:].cpu().double().numpy(), None, None, float(np.float32(1e-6)))
    scale = OB.row_scale(y64)
    v = y64 / scale[:, None]
    got = y[cap - 1:].cpu().double().numpy()
    assert np.all((OB.to_e4m3(v - np.abs(v) * 67 * F) <= got) & (got <= OB.to_e4m3(v + np.abs(v) * 67 * F)))
    assert abs(sc[cap - 1].item() / scale[0] - 1) <= 34 * F
