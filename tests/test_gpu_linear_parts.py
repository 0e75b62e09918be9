"""fp32 outputs of rra_linear_epilogue over a long K are summed in parts of K = 512, whichever kernel the shape takes
(needs a GPU).

The inputs are positive (0.75 to 1.25), so every truncation goes the same way and shows as a bias.  Bound, with f = 2^-23
and S = sum_k a w (the value itself): a product of the tensor core over 16 elements of K truncates the running sum once, by
at most f of it (a single sum over K = 8192, 512 such products, has measured 1e-5 of S: f S / 2 for each product times 0.35,
the mean loss of a truncation in units of f).  Within a part the running sums are S_part j / 32, j = 1 .. 32 (10 % allowed for
the spread of the values): 1.1 x 16.5 f S over all parts.  The parts are added in fp32, off by f / 2 of the running sum each:
1.1 (n + 1) / 4 f S for n = K / 512 parts in a row.  Joining up to 8 shares of K adds 4 f S, and 1 f S is left for the
oracle's inputs of the last addition.  One sum over K = 4096 is off by about 45 f S, over 16384 by 180 f S.
"""
import pytest
import torch

from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu
F = 2.0 ** -23


@pytest.mark.parametrize("cap,K,N", [
    (4, 65536, 64), (16, 16384, 72),                       # few rows
    (17, 16384, 9856), (100, 16384, 19456),                # up to 128 rows, K not shared
    (64, 65536, 264),                                      # and shared by a cluster
    (200, 16384, 9728), (256, 65536, 4096), (256, 32768, 4096), (129, 65536, 264),     # up to 256
    (600, 16384, 256),                                     # in row tiles
    (257, 65536, 520), (1500, 16384, 1032)])               # pairs of SMs
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_long_sums_of_fp32_outputs(cap, K, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(cap + K + N)
    a = (0.75 + 0.5 * torch.rand((cap, K), generator=g, device="cuda")).to(dtype)
    w = (0.75 + 0.5 * torch.rand((N, K), generator=g, device="cuda")).to(dtype)
    c = torch.full((cap, N), float("nan"), device="cuda")
    cu = torch.tensor([0, cap], dtype=torch.int32, device="cuda")
    rra.get_device_error(clear=True)
    rra.linear_epilogue(a, w, cu, 1, c)
    want = torch.empty((cap, N), dtype=torch.float64, device="cuda")
    for n in range(0, N, 1024):
        want[:, n:n + 1024] = a.double() @ w[n:n + 1024].double().t()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    bound = F * (1.1 * 16.5 + 1.1 * (K / 512 + 1) / 4 + 5)
    off = ((c.double() - want).abs() / want).max().item()
    assert off <= bound, f"{off / F:.1f} steps of 2^-23 off, bound {bound / F:.1f}"
