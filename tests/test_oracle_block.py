"""Pins of the block oracle (CPU): torch in fp64, closed forms, invariants."""
import math

import numpy as np
import pytest
import torch

from oracle import block as OB


@pytest.mark.parametrize("act,fn", [
    ("none", lambda x: x), ("relu", torch.relu), ("gelu", torch.nn.functional.gelu),
    ("gelu_tanh", lambda x: torch.nn.functional.gelu(x, approximate="tanh")), ("silu", torch.nn.functional.silu)])
def test_linear_epilogue_against_torch(act, fn):
    g = torch.Generator().manual_seed(1)
    a, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((7, 24), (16, 24)))
    bias, res = torch.randn(16, generator=g, dtype=torch.float64), torch.randn((7, 16), generator=g, dtype=torch.float64)
    want = fn(a @ w.T + bias)[:5] + res[:5]
    assert np.allclose(OB.linear_epilogue(a, w, bias, act, res, 5), want.numpy(), atol=1e-12)


@pytest.mark.parametrize("causal", [True, False])
def test_attend_rows_against_torch(causal):
    g = torch.Generator().manual_seed(2)
    q = torch.randn((9, 6, 16), generator=g, dtype=torch.float64)
    k, v = (torch.randn((9, 2, 16), generator=g, dtype=torch.float64) for _ in range(2))
    last = np.arange(9) if causal else np.full(9, 8)
    o, mag = OB.attend_rows(q, k, v, 0.25, last)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(3, 1).transpose(0, 1), v.repeat_interleave(3, 1).transpose(0, 1),
        is_causal=causal, scale=0.25).transpose(0, 1)
    assert np.allclose(o, want.numpy(), atol=1e-12)
    assert np.all(mag + 1e-12 >= np.abs(o))
    o, _ = OB.attend_rows(q, k, v, 0.25, np.full(9, -1))
    assert np.all(o == 0)


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_closed_forms(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 32))
    f = 10000.0 ** (-np.arange(8) / 8)
    # Position 0 turns nothing; the rotation keeps each pair's length and leaves the tail alone.
    assert np.array_equal(OB.norm_rope(x, [0] * 4, None, 0.0, f, interleaved, 1.0), x)
    y = OB.norm_rope(x, [5, 1, 77, 1000], None, 0.0, f, interleaved, 1.0)
    assert np.array_equal(y[..., 16:], x[..., 16:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # <rotate(q, a), rotate(k, b)> depends on a - b alone.
    u, w = rng.standard_normal((2, 1, 1, 32))
    r = lambda z, p: OB.norm_rope(z, [p], None, 0.0, 10000.0 ** (-np.arange(16) / 16), interleaved, 1.0)[0, 0]
    assert math.isclose(r(u, 9) @ r(w, 4), r(u, 105) @ r(w, 100), rel_tol=1e-9)
    # The norm alone: unit mean square times the weight.
    n = OB.norm_rope(x, None, np.full(32, 2.0), 0.0, None, interleaved, 1.0)
    assert np.allclose((n ** 2).mean(-1), 4.0)
