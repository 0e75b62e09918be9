"""The accuracy that rra.h states for the activations of rra_linear_epilogue, on fp32 outputs (needs a GPU).

One product by 1 makes the activation's argument exact.  GELU: the formula is off by 1.5e-7 of erfc at most (0.75e-7 |x|); its
evaluation in fp32, two approximate operations (one and two units in the last place) and six roundings among it, makes 6e-7 |x|
in all (computed over [-9, 9] in emulation with both approximations off either way), 1e-7 |x| below -3.  SiLU: __expf is off by
2 + 1.17 |x| units, the reciprocal by one, two roundings: (4 + 1.2 |x|) 2^-23 relative below zero, 4 x 2^-23 above plus the
exponential's share e^-x (2 + 1.17 x) 2^-23 <= 2.2 x 2^-23.  tanh-GELU: the same in y, whose own relative error is up to 2.5 x
2^-23.  Results below 2^-126 |x| may be zero.
"""
import numpy as np
import pytest
import torch
from scipy import special

from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu
F = 2.0 ** -23


def _through(x, act, cap, K):
    """act(x) by the kernel that `cap` rows of K take; x fp16 values."""
    out = []
    w = torch.zeros((8, K), dtype=torch.float16, device="cuda")
    w[:, 0] = 1
    for i in range(0, len(x), cap):
        part = x[i:i + cap]
        a = torch.zeros((cap, K), dtype=torch.float16, device="cuda")
        a[:len(part), 0] = part.cuda()
        c = torch.empty((cap, 8), device="cuda")
        rra.linear_epilogue(a, w, torch.tensor([0, len(part)], dtype=torch.int32, device="cuda"), 1, c, act=act)
        assert torch.equal(c[:len(part), 0], c[:len(part), 7])
        out.append(c[:len(part), 0].cpu())
    return torch.cat(out).double().numpy()


@pytest.mark.parametrize("cap,K,step", [(8, 8, 97), (100, 4096, 7), (4000, 8, 1)], ids=["few", "mid", "pair"])
def test_activations_are_as_accurate_as_stated(cap, K, step):
    bits = torch.arange(0, 2 ** 16, step, dtype=torch.int32).to(torch.int16).view(torch.float16)
    x16 = bits[torch.isfinite(bits) & (bits.abs() <= 100)]
    x = x16.double().numpy()
    tiny = 2.0 ** -126 * np.abs(x) + 2.0 ** -149
    got = _through(x16, rra.ACT_GELU, cap, K)
    ref = 0.5 * x * special.erfc(-x / np.sqrt(2))
    tol = np.where(x < -3, 1e-7, 6.5e-7) * np.abs(x) + tiny
    assert np.all(np.abs(got - ref) <= tol)
    got = _through(x16, rra.ACT_SILU, cap, K)
    ref = x * special.expit(x)
    rel = np.where(x < 0, 4 + 1.2 * np.abs(x), 6.2)
    assert np.all(np.abs(got - ref) <= rel * F * np.abs(ref) + tiny)
    got = _through(x16, rra.ACT_GELU_TANH, cap, K)
    y = 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    ref = x * special.expit(y)
    # (1.17 + 2.5) |y| units below zero; above, e^-y |y| <= 0.37 of it.
    rel = np.where(x < 0, 4 + 3.7 * np.abs(y), 4 + 2.2 + 3.7)
    assert np.all(np.abs(got - ref) <= rel * F * np.abs(ref) + tiny)
