"""rra_attend_prompt against the fp64 oracle (needs a GPU); the bound is derived in block_util."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import check_rows, nan_fill
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


def _run(lens, Hq, Hkv, d, dtype, causal, seed, pad=3, scale=None, gain=1.0, rows=None, max_seqlen=None):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    qkv = torch.randn((T + pad, Hq + 2 * Hkv, d), generator=g)
    qkv[:, :Hq] *= gain
    qkv = qkv.to(dtype)
    dev = qkv.cuda()
    nan_fill(dev[T:])                                               # rows behind the last sequence may hold anything
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    o = nan_fill(torch.empty((T + pad, Hq, d), dtype=dtype, device="cuda"))
    scale = d ** -0.5 if scale is None else scale
    rra.get_device_error(clear=True)
    rra.attend_prompt(dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:], cu, len(lens), max_seqlen or max(lens), o,
                      scale=scale, causal=causal)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    got = o.cpu()
    assert bool(torch.isnan(got[T:].float()).all()), "rows past the last sequence were written"
    a = 0
    for n in lens:
        last = np.arange(n) if causal else np.full(n, n - 1)
        pick = None if rows is None else np.unique(np.clip(rows, 0, n - 1))
        if n:
            check_rows(got[a:a + n], qkv[a:a + n, :Hq], qkv[a:a + n, Hq:Hq + Hkv], qkv[a:a + n, Hq + Hkv:], scale, last,
                       dtype, pick)
        a += n
    return got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 300, 385, 513])
def test_attend_prompt_lengths(n, dtype, d, causal):
    _run([n], 2, 1, d, dtype, causal, seed=n + d)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (12, 12, 64), (7, 7, 128), (8, 2, 128), (6, 2, 64), (8, 1, 128)])
def test_attend_prompt_heads_and_ragged_batches(Hq, Hkv, d, causal):
    _run([130, 0, 1, 257, 0, 64, 33, 0], Hq, Hkv, d, torch.bfloat16, causal, seed=Hq + d)
    _run([0, 0, 5], Hq, Hkv, d, torch.float16, causal, seed=1)
    _run([0, 1], Hq, Hkv, d, torch.float16, causal, seed=2, pad=0, max_seqlen=5000)
    _run([130, 0, 1, 257, 33], Hq, Hkv, d, torch.bfloat16, causal, seed=3, max_seqlen=100000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain,scale", [(8.0, None), (30.0, None), (1.0, 1e-4), (1.0, 3.0)])
def test_attend_prompt_score_ranges(d, gain, scale):
    """Flat and peaked softmaxes; the running maximum moves by large steps."""
    _run([400], 2, 2, d, torch.bfloat16, True, seed=5, gain=gain, scale=scale)
    _run([400], 2, 2, d, torch.float16, False, seed=6, gain=gain, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_prompt_rising_scores(d):
    """Keys that grow along the sequence: the row maximum rises block after block, far past any fixed reference."""
    n, dtype = 1100, torch.bfloat16
    g = torch.Generator().manual_seed(2)
    q, v = torch.ones((n, 1, d)).to(dtype), torch.randn((n, 1, d), generator=g).to(dtype)
    k = (torch.arange(n)[:, None, None] / 40.0 * torch.ones((1, 1, d))).to(dtype)
    for kk in (k, k.flip(0), -k):
        o = torch.empty((n, 1, d), dtype=dtype, device="cuda")
        kk = kk.contiguous()
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        for causal in (True, False):
            rra.attend_prompt(q.cuda(), kk.cuda(), v.cuda(), cu, 1, n, o, scale=d ** -0.5, causal=causal)
            last = np.arange(n) if causal else np.full(n, n - 1)
            check_rows(o.cpu(), q, kk, v, d ** -0.5, last, dtype, np.arange(0, n, 7))


def test_attend_prompt_long():
    """A few thousand keys, sampled rows."""
    rows = np.array([0, 1, 127, 128, 300, 1023, 2047, 2048, 2500, 3998, 3999])
    _run([4000, 17, 2049], 4, 1, 128, torch.bfloat16, True, seed=3, rows=rows)
    _run([4000, 17, 2049], 3, 3, 64, torch.float16, False, seed=4, rows=rows)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_prompt_keys_out_of_sight(d):
    """Infinite and NaN keys in the future of a row do not reach it; other sequences' rows hold anything."""
    n, dtype = 300, torch.bfloat16
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn((2 * n, 2, d), generator=g).to(dtype) for _ in range(3))
    cu = torch.tensor([n, 2 * n], dtype=torch.int32, device="cuda")
    k2, v2 = k.clone(), v.clone()
    k2[:n], v2[:n] = float("nan"), float("nan")                      # rows before the sequence
    k2[n + 200], k2[n + 250] = float("inf"), float("nan")
    o, o2 = (nan_fill(torch.empty((2 * n, 2, d), dtype=dtype, device="cuda")) for _ in range(2))
    rra.attend_prompt(q.cuda(), k.cuda(), v.cuda(), cu, 1, n, o, scale=0.1)
    rra.attend_prompt(q.cuda(), k2.cuda(), v2.cuda(), cu, 1, n, o2, scale=0.1)
    torch.cuda.synchronize()
    assert torch.equal(o[n:n + 200], o2[n:n + 200])
    assert bool(torch.isnan(o2[:n].float()).all())                   # not written
    assert bool(torch.isnan(o2[n + 250:].float()).all())


def test_attend_prompt_bad_lengths_are_reported_and_skipped():
    n, d = 64, 128
    q, k, v = (torch.randn((3 * n, 2, d), device="cuda").bfloat16() for _ in range(3))
    for cu, S, code, good in (([0, n, 3 * n], n, rra.DEVERR_SEQ_TOO_LONG, (0, n)),
                              ([n, 0, n], n, rra.DEVERR_SEQ_NEGATIVE, (0, n)),
                              ([2 * n, 3 * n, 4 * n], n, rra.DEVERR_INDEX_RANGE, (2 * n, 3 * n)),
                              ([-n, 0, n], n, rra.DEVERR_INDEX_RANGE, (0, n))):
        o = nan_fill(torch.empty_like(q))
        rra.get_device_error(clear=True)
        rra.attend_prompt(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), 2, S, o, scale=0.1)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == code
        a, b = good
        check_rows(o[a:b].cpu(), q[a:b].cpu(), k[a:b].cpu(), v[a:b].cpu(), 0.1, np.arange(n), torch.bfloat16)
        rest = torch.ones(3 * n, dtype=torch.bool, device="cuda")
        rest[a:b] = False
        assert bool(torch.isnan(o[rest].float()).all())


def test_attend_prompt_rows_past_32_bits():
    """Rows whose offsets pass 2^32 elements; o's pass 2^31."""
    d, n = 128, 200
    cap = (1 << 24) + 64                                             # o: 2^24 rows x 128 = 2^31 elements
    stride = 3 * d
    big = torch.empty((cap, 3, d), dtype=torch.bfloat16, device="cuda")   # 6.4e9 elements
    g = torch.Generator().manual_seed(1)
    x = torch.randn((n, 3, d), generator=g).to(torch.bfloat16)
    big[cap - n:] = x.cuda()
    assert (cap - n) * stride > 2 ** 32
    o = torch.zeros((cap, 1, d), dtype=torch.bfloat16, device="cuda")
    rra.get_device_error(clear=True)
    rra.attend_prompt(big[:, :1], big[:, 1:2], big[:, 2:], torch.tensor([cap - n, cap], dtype=torch.int32, device="cuda"),
                      1, n, o, scale=0.1)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    check_rows(o[cap - n:].cpu(), x[:, :1], x[:, 1:2], x[:, 2:], 0.1, np.arange(n), torch.bfloat16)
    assert bool((o[:cap - n] == 0).all())


def test_attend_prompt_many_short_sequences_and_a_loose_bound():
    """Thousands of sequences of 0 to 5 rows; a max_seqlen far above the longest costs nothing."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 6, 5000)
    T, d, dtype = int(lens.sum()), 64, torch.float16
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn((T, 1, d), generator=g).to(dtype) for _ in range(3))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    outs = []
    for S in (5, 1 << 30):
        o = nan_fill(torch.empty((T, 1, d), dtype=dtype, device="cuda"))
        rra.get_device_error(clear=True)
        rra.attend_prompt(q.cuda(), k.cuda(), v.cuda(), cu, len(lens), S, o, scale=0.125)
        torch.cuda.synchronize()
        assert rra.get_device_error() == 0
        outs.append(o.cpu())
    assert torch.equal(outs[0], outs[1])
    a = 0
    for n in lens:
        if n:
            check_rows(outs[0][a:a + n], q[a:a + n], k[a:a + n], v[a:a + n], 0.125, np.arange(n), dtype)
        a += n


def test_attend_prompt_repeats_bit_for_bit_and_in_graphs():
    lens, Hq, Hkv, d = [700, 1, 130], 8, 2, 128
    T = sum(lens)
    q, k, v = (torch.randn((T, h, d), device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 700, 701, T], dtype=torch.int32, device="cuda")
    call = lambda o: rra.attend_prompt(q, k, v, cu, 3, 700, o, scale=0.09)
    outs = [torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    call(outs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(outs[1])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[2])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_prompt_many_units(d, causal):
    """More units than SMs, whole: ragged tiles end to end, one call long enough that every CTA takes several."""
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(0, 300, 24)] + [127, 128, 129, 255, 256, 257, 1, 2]
    _run(lens, 12, 12, d, torch.bfloat16, causal, seed=d)
    _run(lens, 8, 4, d, torch.float16, causal, seed=d + 1)


@pytest.mark.parametrize("d,Hq,Hkv,causal,lens", [
    (128, 8, 1, True, [4096]), (128, 16, 4, True, [2047]), (64, 12, 4, False, [3900]), (64, 12, 12, True, [3841, 1]),
    (128, 12, 12, False, [100, 3009, 128, 0, 129])])
def test_attend_prompt_keys_split_over_several_rounds(d, Hq, Hkv, causal, lens):
    """Few long prompts: both tiles of a unit are the same rows, and CTAs take several units, some of one block."""
    rows = np.array([0, 1, 126, 127, 128, 129, 255, 256, 1000, 2046, 2047, 3008, 3840, 3899, 4095])
    _run(lens, Hq, Hkv, d, torch.bfloat16, causal, seed=Hq, rows=rows)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_prompt_blocks_of_infinite_scores(d, dtype):
    """Every other block of 128 keys at -inf (scores -inf, weights 0), either way round; and scores far apart from block to block."""
    n = 700
    g = torch.Generator().manual_seed(9)
    q, v = torch.rand((n, 2, d), generator=g).to(dtype) + 0.5, torch.randn((n, 2, d), generator=g).to(dtype)
    k = torch.randn((n, 2, d), generator=g).to(dtype)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    block = torch.arange(n) // 128
    for odd in (0, 1):
        kk = k.clone()
        kk[block % 2 == odd, :, 3] = float("-inf")
        o = nan_fill(torch.empty((n, 2, d), dtype=dtype, device="cuda"))
        rra.attend_prompt(q.cuda(), kk.cuda(), v.cuda(), cu, 1, n, o, scale=0.1, causal=False)
        seen = block % 2 != odd
        m = int(seen.sum())
        check_rows(o.cpu()[:m], q[:m], k[seen], v[seen], 0.1, np.full(m, m - 1), dtype)
        # Causal: rows of block 0 that see -inf alone sum to nothing and come out as zeros.
        rra.attend_prompt(q.cuda(), kk.cuda(), v.cuda(), cu, 1, n, o, scale=0.1)
        torch.cuda.synchronize()
        got = o.cpu().float()
        assert bool(torch.isfinite(got).all())
        if odd == 0:
            assert bool((got[:128] == 0).all()) and bool((got[128:] != 0).any())
        kk = k.clone()
        kk[block % 2 == odd] *= 40.0
        rra.attend_prompt(q.cuda(), kk.cuda(), v.cuda(), cu, 1, n, o, scale=0.1)
        check_rows(o.cpu(), q, kk, v, 0.1, np.arange(n), dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_prompt_overlapping_sequences(d):
    """Offsets that go back make more units than the capacity suggests: each valid sequence is answered, the rest reported."""
    n, S = 300, 40
    q, k, v = (torch.randn((n, 4, d), device="cuda").bfloat16() for _ in range(3))
    cu = torch.tensor([0, n] * S, dtype=torch.int32, device="cuda")
    o = nan_fill(torch.empty_like(q))
    rra.get_device_error(clear=True)
    rra.attend_prompt(q, k, v, cu, 2 * S - 1, n, o, scale=0.1)
    torch.cuda.synchronize()
    assert rra.get_device_error(clear=True) == rra.DEVERR_SEQ_NEGATIVE
    check_rows(o.cpu(), q.cpu(), k.cpu(), v.cpu(), 0.1, np.arange(n), torch.bfloat16)
