"""rra_attend_paged against the fp64 oracle (needs a GPU); the bound is derived in block_util."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import check_rows, nan_fill
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Paged:
    """Sequences of `new` tokens on top of caches of `kv` keys in all, in pages in a random order; what no sequence uses is
    NaN, and table entries behind the last page point outside the pool."""

    def __init__(self, new, kv, Hq, Hkv, d, page, dtype, seed, gain=1.0, joint=False, gap=0, q_pad=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.dtype, self.page, self.d = new, kv, dtype, page, d
        need = [-(-m // page) for m in kv]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g).tolist()
        width = max(max(need), 1) + 2
        table = np.full((len(kv), width), 2 ** 31 - 1, np.int32)
        pool = nan_fill(torch.empty((pages, 2, page, Hkv, d), dtype=dtype))
        self.k, self.v = [], []
        for b, m in enumerate(kv):
            ids = [order.pop() for _ in range(need[b])]
            table[b, :need[b]] = ids
            k, v = (torch.randn((m, Hkv, d), generator=g).to(dtype) for _ in range(2))
            for i, p in enumerate(ids):
                part = slice(i * page, min(m, (i + 1) * page))
                pool[p, 0, :part.stop - part.start], pool[p, 1, :part.stop - part.start] = k[part], v[part]
            self.k.append(k)
            self.v.append(v)
        self.table = torch.from_numpy(table).cuda()
        if joint:
            dev = pool.cuda()
            self.kd, self.vd = dev[:, 0], dev[:, 1]
        else:
            self.kd, self.vd = pool[:, 0].contiguous().cuda(), pool[:, 1].contiguous().cuda()
        self.at = gap + np.concatenate([[0], np.cumsum(new)])
        self.cap = int(self.at[-1]) + gap
        self.q = (torch.randn((self.cap, Hq + q_pad, d), generator=g) * gain).to(dtype)
        nan_fill(self.q[:gap])
        nan_fill(self.q[int(self.at[-1]):])
        self.q_pad, self.Hq = q_pad, Hq
        self.qd = self.q.cuda()[:, :Hq]
        self.o = nan_fill(torch.empty((self.cap, Hq, d), dtype=dtype, device="cuda"))

    def call(self, scale=None, max_new=None, max_kv=None, stream=None):
        rra.attend_paged(self.qd, self.kd, self.vd, self.table, _ints(self.kv), _ints(self.at), len(self.kv),
                         max_new or max(max(self.new), 1), max_kv or max(max(self.kv), 1), self.o,
                         scale=scale or self.d ** -0.5, stream=stream)

    def check(self, scale=None, rows=None, seqs=None):
        torch.cuda.synchronize()
        got = self.o.cpu()
        for b in range(len(self.kv)) if seqs is None else seqs:
            n, m = self.new[b], self.kv[b]
            sl = slice(int(self.at[b]), int(self.at[b + 1]))
            last = m - n + np.arange(n)
            pick = None if rows is None else np.unique(np.clip(rows, 0, max(n - 1, 0)))
            if n:
                k, v = (self.k[b], self.v[b]) if m else (torch.zeros((1, *self.k[b].shape[1:])),) * 2
                check_rows(got[sl], self.q[sl, :self.Hq], k, v, scale or self.d ** -0.5, last, self.dtype, rows=pick)
            for i in range(min(n, max(0, n - m))):
                assert bool((got[sl][i] == 0).all()), "a row that sees nothing is zero"
        assert bool(torch.isnan(got[:int(self.at[0])].float()).all() and torch.isnan(got[int(self.at[-1]):].float()).all())

    def run(self, rows=None, **kw):
        rra.get_device_error(clear=True)
        self.call(**kw)
        torch.cuda.synchronize()
        assert rra.get_device_error() == 0
        self.check(rows=rows)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 12), (8, 2), (7, 1), (14, 2), (32, 2), (40, 1)])
def test_attend_paged_heads(Hq, Hkv, d, dtype):
    kv = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100]
    Paged([1] * len(kv), kv, Hq, Hkv, d, 16, dtype, seed=Hq + d).run()
    Paged([min(9, m) for m in kv], kv, Hq, Hkv, d, 32, dtype, seed=Hq + d, joint=True, gap=3).run()


@pytest.mark.parametrize("page", [16, 32, 48, 64, 112, 128, 256, 1024])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_paged_page_sizes(page, d):
    """Lengths around the ends of pages and of the kernels' blocks, one new token, a few and whole chunks."""
    kv = [page - 1, page, page + 1, 2 * page, 127, 128, 129, 255, 257, 300]
    for n in (1, 3, 40, 140):
        Paged([min(n, m) for m in kv], kv, 4, 2, d, page, torch.bfloat16, seed=page + n, joint=n == 3).run()


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (6, 2, 128), (8, 1, 128), (7, 1, 64), (12, 12, 64), (16, 1, 128)])
@pytest.mark.parametrize("n", [2, 17, 64, 127, 128, 129, 300])
def test_attend_paged_chunks(n, Hq, Hkv, d):
    """Chunks on caches of all lengths; more new tokens than keys leave the first rows without any."""
    Paged([n] * 6, [0, 1, n - 1, n, n + 1, n + 333], Hq, Hkv, d, 32, torch.bfloat16, seed=n, gap=2, q_pad=3).run()


@pytest.mark.parametrize("Hq,Hkv", [(64, 1), (128, 1), (129, 1), (300, 2)])
def test_attend_paged_large_groups(Hq, Hkv):
    """Up to a head a row of a tile, and more heads to a group than a tile has rows."""
    Paged([3, 0, 1, 20], [30, 5, 200, 20], Hq, Hkv, 64, 16, torch.bfloat16, seed=Hq).run()


def test_attend_paged_mixed_batch():
    new = [1, 0, 200, 1, 33, 1, 1, 130, 0, 5, 1]
    kv = [1000, 50, 777, 1, 33, 2049, 0, 129, 0, 400, 16]
    for Hq, Hkv, d, page in ((8, 2, 128, 16), (6, 6, 64, 48)):
        Paged(new, kv, Hq, Hkv, d, page, torch.bfloat16, seed=d, joint=True, gap=5).run()
        Paged(new, kv, Hq, Hkv, d, page, torch.float16, seed=d).run(max_new=4000, max_kv=2049)


@pytest.mark.parametrize("B", [1, 3, 40])
@pytest.mark.parametrize("most", [1, 64, 1000, 9000])
def test_attend_paged_batches_and_lengths(B, most):
    rng = np.random.default_rng(B + most)
    kv = [most] + [int(x) for x in rng.integers(0, most + 1, B - 1)]
    Paged([1] * B, kv, 4, 1, 128, 64, torch.bfloat16, seed=B).run()


@pytest.mark.parametrize("Hq,Hkv,d,page", [(8, 2, 128, 64), (1, 1, 64, 16), (12, 6, 64, 48)])
def test_attend_paged_tokens_by_tiles(Hq, Hkv, d, page):
    """Next tokens with loose or long bounds go as tiles too: contexts of very different lengths, some empty."""
    kv = [9000, 0, 1, 100, 17, 4095, 4096, 4097, 128, 0, 33, 2000] * 3
    p = Paged([1, 1, 1, 0] * 9, kv, Hq, Hkv, d, page, torch.bfloat16, seed=Hq, gap=1, joint=True)
    p.table = torch.cat([p.table, p.table.new_full((36, (1 << 20) // page), -7)], 1)
    p.run(max_kv=1 << 20)


@pytest.mark.parametrize("B", [257, 700])
def test_attend_paged_many_sequences(B):
    """More sequences than a CTA has threads, with rows and without."""
    rng = np.random.default_rng(B)
    new = [int(x) for x in rng.choice([0, 0, 1, 1, 1, 9, 40], B)]
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 90, B))]
    Paged(new, kv, 4, 2, 64, 16, torch.bfloat16, seed=B).run()
    new = [0] * B
    new[B - 2] = 70
    Paged(new, kv[:B - 2] + [500, 0], 4, 2, 128, 16, torch.bfloat16, seed=B).run()


def test_attend_paged_thousands_of_sequences():
    """A batch of thousands by tiles, most of them without new tokens; some of them looked at."""
    rng = np.random.default_rng(1)
    B = 6000
    new = [int(x) for x in rng.choice([0, 0, 0, 1, 2], B)]
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 60, B))]
    new[4321], kv[4321] = 50, 700
    p = Paged(new, kv, 4, 2, 64, 16, torch.bfloat16, seed=2)
    rra.get_device_error(clear=True)
    p.call()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    p.check(seqs=[0, 1, 2, 255, 256, 257, 511, 512, 3000, 4320, 4321, 4322, B - 2, B - 1] + list(range(100, 140)))
    assert bool(torch.isfinite(p.o.float()).all())


@pytest.mark.parametrize("n,m", [(5, 9000), (48, 20000), (150, 5000), (600, 3000), (1, 40000)])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_paged_long_caches(n, m, d):
    """Few rows over many keys: the keys are split; rows picked here and there."""
    Paged([n, min(n, 7)], [m, 700], 8, 2, d, 64, torch.bfloat16, seed=n).run(rows=np.linspace(0, n - 1, 9).astype(int))


@pytest.mark.parametrize("gain", [8.0, 40.0])
def test_attend_paged_peaked(gain):
    for n in (1, 2, 70):
        Paged([n, n], [3000, 100], 4, 2, 64, 32, torch.float16, seed=3, gain=gain).run()
        Paged([n, n], [3000, 100], 4, 2, 128, 16, torch.bfloat16, seed=4, gain=gain).run()


def test_attend_paged_keys_infinite_or_nan_touch_only_the_rows_that_see_them():
    for n in (4, 200):
        p = Paged([n], [n + 50], 2, 1, 64, 16, torch.bfloat16, seed=n)
        j = n + 48                                                   # seen by the last two rows only
        p.kd[int(p.table[0, j // 16]), j % 16] = float("nan")
        p.call()
        torch.cuda.synchronize()
        assert bool(torch.isnan(p.o[n - 2:n].float()).all())
        full = p.o.clone()
        p.o[n - 2:n] = 0
        last = 50 + np.arange(n)
        check_rows(full[:n - 2].cpu(), p.q[:n - 2], p.k[0], p.v[0], 64 ** -0.5, last[:n - 2], torch.bfloat16)


def test_attend_paged_shared_pages():
    """Two sequences whose tables start with the same pages (a common prefix)."""
    p = Paged([3, 30], [64, 128], 4, 2, 128, 32, torch.bfloat16, seed=9)
    p.table[1, :2] = p.table[0, :2]
    p.k[1][:64], p.v[1][:64] = p.k[0], p.v[0]
    p.run()


def test_attend_paged_pool_past_32_bits():
    """A pool whose offsets pass 2^32 elements; a page at its far end is read, by one token and by a chunk."""
    page, Hkv, d = 256, 8, 128
    pages = (1 << 14) + 9                                            # 4.3e9 elements each
    kd, vd = (torch.empty((pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    m = 400
    k, v = (torch.randn((m, Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
    ids = [pages - 1, pages - 2]
    for t, x in ((kd, k), (vd, v)):
        t[ids[0]] = x[:256].cuda()
        t[ids[1], :144] = x[256:].cuda()
    for n in (1, 90):
        q = torch.randn((n, 16, d), generator=g).to(torch.bfloat16)
        o = nan_fill(torch.empty((n, 16, d), dtype=torch.bfloat16, device="cuda"))
        rra.attend_paged(q.cuda(), kd, vd, _ints([ids]), _ints([m]), _ints([0, n]), 1, n, m, o, scale=0.09)
        torch.cuda.synchronize()
        check_rows(o.cpu(), q, k, v, 0.09, m - n + np.arange(n), torch.bfloat16)


@pytest.mark.parametrize("n", [1, 5, 150])
def test_attend_paged_bad_lengths_and_pages_are_reported(n):
    """A sequence that is not as declared is not written, a page outside the pool is reported; the others are right."""
    def fresh():
        p = Paged([n, n, n], [n + 20, n + 33, n + 70], 4, 2, 64, 16, torch.bfloat16, seed=n)
        rra.get_device_error(clear=True)
        return p

    for bad, code in ((-1, rra.DEVERR_SEQ_NEGATIVE), (n + 71, rra.DEVERR_SEQ_TOO_LONG)):
        p = fresh()
        right, p.kv = p.kv, [p.kv[0], bad, p.kv[2]]
        p.call(max_kv=n + 70)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == code
        assert bool(torch.isnan(p.o[n:2 * n].float()).all())
        p.kv = right
        p.check(seqs=[0, 2])
    for at, code in (([0, n, n - 1, 3 * n], rra.DEVERR_SEQ_NEGATIVE), ([0, n, 2 * n, 3 * n + 1], rra.DEVERR_SEQ_TOO_LONG)):
        p = fresh()
        right, p.at = p.at, np.asarray(at)
        p.call(max_new=n)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) in (code, rra.DEVERR_SEQ_TOO_LONG)
        p.at = right
        p.check(seqs=[0])
    p = fresh()
    right, p.at = p.at, np.asarray([0, n, 2 * n, 3 * n + 1])
    p.call(max_new=n + 1)
    torch.cuda.synchronize()
    assert rra.get_device_error(clear=True) == (rra.DEVERR_INDEX_RANGE if n + 1 <= p.cap else rra.DEVERR_SEQ_TOO_LONG)
    p.at = right
    p.check(seqs=[0, 1])
    for entry in (-1, p.kd.shape[0]):
        p = fresh()
        p.kd.nan_to_num_(0.0), p.vd.nan_to_num_(0.0)                 # page 0 is read instead: something finite
        p.table[1, 1] = entry
        p.call()
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == rra.DEVERR_INDEX_RANGE
        p.check(seqs=[0, 2])


@pytest.mark.parametrize("new,kv", [([1, 1], [6000, 1234]), ([100, 1], [6000, 1234]), ([700, 300], [800, 300])])
def test_attend_paged_repeats_bit_for_bit_and_in_two_graphs(new, kv):
    """Nothing is shared between calls: two captured graphs replayed in turn and at once give the eager result."""
    ps = [Paged(new, kv, 8, 2, 128, 64, torch.bfloat16, seed=s) for s in range(2)]
    for p in ps:
        p.lens, p.cu = _ints(p.kv), _ints(p.at)

    def call(p, o):
        rra.attend_paged(p.qd, p.kd, p.vd, p.table, p.lens, p.cu, 2, max(new), max(kv), o, scale=0.09)

    want, got = ([torch.empty_like(p.o) for p in ps] for _ in range(2))
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for p, o in zip(ps, want):
        call(p, o)
    torch.cuda.synchronize()
    for p, o in zip(ps, got):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(p, o)
        graphs.append(gr)
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
