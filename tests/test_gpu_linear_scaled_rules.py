"""rra_linear_scaled on both sides of the rules that choose its kernels, and at its most rows (needs a GPU).

Operands are whole numbers and scales powers of two: every sum is exact in fp32, so results are the formula's, rounded once.
"""
from __future__ import annotations

import pytest
import torch

from block_util import nan_fill
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


def _run(T, cap, K, N, out, residual, seed, rows=None):
    """rows: the rows looked at (None: all); without `residual` a ReLU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ints = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").to(torch.float16)
    a, w = ints(cap, K).to(E4), ints(N, K).to(E4)
    sa = 2.0 ** -(torch.arange(cap, device="cuda") % 3).float()
    sw = 2.0 ** -(8 + torch.arange(N, device="cuda") % 3).float()
    b = ints(N).float()
    c = nan_fill(torch.empty((cap, N), dtype=out, device="cuda"))
    if residual:
        c.copy_(ints(cap, N))
        r = c.clone()
    nan_fill(a[T:])
    rra.get_device_error(clear=True)
    rra.linear_scaled(a, sa, w, sw, torch.tensor([0, T], dtype=torch.int32, device="cuda"), 1, c, bias=b,
                      act=rra.ACT_NONE if residual else rra.ACT_RELU, residual=c if residual else None)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    at = torch.arange(T, device="cuda") if rows is None else torch.as_tensor(rows, device="cuda")
    a64 = a.view(torch.uint8)[at].view(E4).to(torch.float64) * sa[at, None].double()
    for n in range(0, N, 4096):
        m = min(N, n + 4096)
        want = a64 @ (w[n:m].to(torch.float64) * sw[n:m, None].double()).t() + b[n:m].double()
        want = want + r[at, n:m].double() if residual else want.clamp(min=0.0)
        assert torch.equal(c[at, n:m], want.to(out)), f"columns {n} to {m}"
    if residual:
        assert torch.equal(c[T:], r[T:])
    else:
        assert bool(torch.isnan(c[T:].float()).all()), "rows past T were written"


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("cap", [1, 8, 9, 16])
@pytest.mark.parametrize("K", [64, 272, 2064])
def test_80_columns_an_sm(cap, K):
    """A CTA for 16 columns of a few rows up to there, tiles of 128 columns beyond."""
    for N in (80 * _sms(), 80 * _sms() + 8):
        for out in (torch.bfloat16, torch.float32):
            _run(cap, cap, K, N, out, cap % 2 == 0, seed=cap + K + N)


@pytest.mark.parametrize("N", [6144, 6152])
def test_weights_of_24_megabytes(N):
    for cap in (8, 9, 16):
        _run(cap - 1, cap, 4096, N, torch.bfloat16, True, seed=cap + N)


@pytest.mark.parametrize("T,cap,K,N", [(24, 24, 4096, 65536), (49, 64, 4096, 32768), (64, 64, 8192, 24472), (96, 96, 8192, 30472),
                                       (101, 112, 16384, 30472), (112, 112, 16384, 33480), (128, 128, 16384, 33480)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
def test_tens_of_rows_in_several_rounds(T, cap, K, N, out):
    """Two CTAs an SM for all of these on 152 SMs but the last, where pairs of SMs have the tiles."""
    _run(T, cap, K, N, out, True, seed=T)
    _run(T, cap, K, N, out, False, seed=T + 1)


def test_the_most_rows():
    cap = 65535 * 128
    rows = [0, 1, 255, 256, 1 << 22, cap - 300, cap - 129, cap - 128, cap - 2]
    _run(cap - 1, cap, 16, 8, torch.bfloat16, False, seed=1, rows=rows)
    _run(cap - 1, cap, 16, 8, torch.float32, True, seed=2, rows=rows)
