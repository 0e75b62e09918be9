"""rra_attend_cache against the fp64 oracle (needs a GPU); the bound is derived in block_util."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import check_rows, nan_fill
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


def _run(lens, cap, nq, Hq, Hkv, d, dtype, seed, gain=1.0, q_pad=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    q = (torch.randn((B * nq, Hq + q_pad, d), generator=g) * gain).to(dtype)
    k, v = (torch.randn((B, cap, Hkv, d), generator=g).to(dtype) for _ in range(2))
    kd, vd = k.cuda(), v.cuda()
    for b, n in enumerate(lens):
        nan_fill(kd[b, n:])                                         # rows not in use may hold anything
        nan_fill(vd[b, n:])
    o = nan_fill(torch.empty((B * nq, Hq, d), dtype=dtype, device="cuda"))
    rra.get_device_error(clear=True)
    rra.attend_cache(q.cuda()[:, :Hq], kd, vd, torch.tensor(lens, dtype=torch.int32, device="cuda"), o, scale=d ** -0.5)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    got = o.cpu()
    for b, n in enumerate(lens):
        sl = slice(b * nq, (b + 1) * nq)
        last = n - nq + np.arange(nq)
        check_rows(got[sl], q[sl, :Hq], k[b, :max(n, 1)], v[b, :max(n, 1)], d ** -0.5, last, dtype)
        for i in range(nq):
            if last[i] < 0:
                assert bool((got[b * nq + i] == 0).all()), "a row that sees nothing is zero"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 12), (8, 2), (7, 1), (14, 2), (32, 2), (40, 1)])
def test_attend_cache_heads(Hq, Hkv, d, dtype):
    _run([0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100], 100, 1, Hq, Hkv, d, dtype, seed=Hq + d)


@pytest.mark.parametrize("nq", [1, 2, 3, 5, 16, 33, 64])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (6, 2, 128), (8, 1, 128)])
def test_attend_cache_several_new_tokens(nq, Hq, Hkv, d):
    """More new tokens than keys leave the first rows without any."""
    _run([0, 1, nq - 1, nq, nq + 1, 129, 200], 200, nq, Hq, Hkv, d, torch.bfloat16, seed=nq)


@pytest.mark.parametrize("B", [1, 3, 40])
@pytest.mark.parametrize("cap", [1, 64, 1000, 9000])
def test_attend_cache_batches_and_lengths(B, cap):
    rng = np.random.default_rng(B + cap)
    lens = [cap] + [int(x) for x in rng.integers(0, cap + 1, B - 1)]
    _run(lens, cap, 1, 4, 1, 128, torch.bfloat16, seed=B, q_pad=2)


@pytest.mark.parametrize("gain", [8.0, 40.0])
def test_attend_cache_peaked(gain):
    _run([3000, 40], 3000, 1, 4, 2, 64, torch.float16, seed=3, gain=gain)
    _run([3000, 40], 3000, 2, 4, 2, 128, torch.bfloat16, seed=4, gain=gain)


def test_attend_cache_past_32_bits():
    """A cache whose offsets pass 2^32 elements; the last sequence is read."""
    B, cap, Hkv, d = 3, (1 << 21) + 16, 8, 128                      # 6.4e9 elements
    k, v = (torch.empty((B, cap, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 700
    g = torch.Generator().manual_seed(1)
    kk, vv = (torch.randn((n, Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((B, 16, d), generator=g).to(torch.bfloat16)
    k[2, :n], v[2, :n] = kk.cuda(), vv.cuda()
    o = torch.empty((B, 16, d), dtype=torch.bfloat16, device="cuda")
    rra.attend_cache(q.cuda(), k, v, torch.tensor([0, 0, n], dtype=torch.int32, device="cuda"), o, scale=0.09)
    torch.cuda.synchronize()
    assert bool((o[:2] == 0).all())
    check_rows(o[2:].cpu(), q[2:], kk, vv, 0.09, [n - 1], torch.bfloat16)
    # and at the far end of one sequence
    k[0, :] = 0
    v[0, :] = 0
    v[0, cap - 1] = 1.0
    rra.attend_cache(q.cuda(), k, v, torch.tensor([cap, 0, 0], dtype=torch.int32, device="cuda"), o, scale=0.09)
    torch.cuda.synchronize()
    assert bool((o[0].float() * cap - 1).abs().max() <= 2.0 ** -7)      # the mean of one 1 among cap zeros, rounded


def test_attend_cache_bad_lengths_are_reported():
    B, cap, d = 3, 50, 64
    k, v = (torch.randn((B, cap, 2, d), device="cuda").half() for _ in range(2))
    q = torch.randn((B, 4, d), device="cuda").half()
    for bad, code in ((-1, rra.DEVERR_SEQ_NEGATIVE), (cap + 1, rra.DEVERR_SEQ_TOO_LONG)):
        o = nan_fill(torch.empty_like(q))
        rra.get_device_error(clear=True)
        rra.attend_cache(q, k, v, torch.tensor([20, bad, cap], dtype=torch.int32, device="cuda"), o, scale=0.125)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == code
        assert bool(torch.isnan(o[1].float()).all())
        for b, n in ((0, 20), (2, cap)):
            check_rows(o[b:b + 1].cpu(), q[b:b + 1].cpu(), k[b, :n].cpu(), v[b, :n].cpu(), 0.125, [n - 1], torch.float16)


def test_attend_cache_repeats_bit_for_bit_and_in_two_graphs():
    """Nothing is shared between calls: two captured graphs replayed in turn and at once give the eager result."""
    B, cap, Hq, Hkv, d = 2, 6000, 8, 2, 128
    k, v = (torch.randn((B, cap, Hkv, d), device="cuda").bfloat16() for _ in range(2))
    q = [torch.randn((B, Hq, d), device="cuda").bfloat16() for _ in range(2)]
    lens = torch.tensor([6000, 1234], dtype=torch.int32, device="cuda")
    call = lambda i, o: rra.attend_cache(q[i], k, v, lens, o, scale=0.09)
    want = [torch.empty_like(q[0]) for _ in range(2)]
    got = [torch.empty_like(q[0]) for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        call(i, want[i])
    torch.cuda.synchronize()
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(i, got[i])
        graphs.append(gr)
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(want[i], got[i])
