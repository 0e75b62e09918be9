"""The row norm, the 8-bit layer and the attention over pages as a serving step uses them (needs a GPU): together with the
block's other operators, on streams, in graphs, with a bound error word, through both marshalling paths, and with waits that
run out."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from block_util import F, check_rows, half_step, nan_fill
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu
E4, BF = torch.float8_e4m3fn, torch.bfloat16


def _ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _eight(w):
    s = w.abs().amax(1) / 448
    return (w / s[:, None]).to(E4), s


def _np(t):
    return t.float().cpu().double().numpy()


def test_chunks_then_tokens_through_a_block():
    """Two steps of a batch: chunks of three prompts, then the rest of one, a token of another, nothing of the third.
    Each operator's output is checked against the oracle on what it was given, as it lies in the buffers."""
    g = torch.Generator().manual_seed(5)
    C, Hq, Hkv, d, page, hidden = 320, 8, 2, 128, 32, 528
    W = (Hq + 2 * Hkv) * d
    wqkv, sqkv = (t.cuda() for t in _eight(torch.randn((W, C), generator=g) / np.sqrt(C)))
    wup, sup = (t.cuda() for t in _eight(torch.randn((hidden, C), generator=g) / np.sqrt(C)))
    wo = (torch.randn((C, Hq * d), generator=g) / np.sqrt(Hq * d)).to(BF).cuda()
    n1, n2 = (1 + 0.1 * torch.randn((2, C), generator=g)).cuda()
    nq, nk = (1 + 0.1 * torch.randn((2, d), generator=g)).cuda()
    inv_freq = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()
    pool = torch.full((13, 2, page, Hkv, d), float("nan"), dtype=BF, device="cuda")
    kp, vp = pool[:, 0], pool[:, 1]
    slots = pool.view(-1, Hkv, d)                              # row (2 p + kv) * page + r
    table = np.array([[3, 9, 1, -1], [7, -1, -1, -1], [12, 0, 5, 2]], np.int32)
    have = np.zeros(3, int)
    rra.get_device_error(clear=True)
    for new in ([70, 20, 40], [1, 0, 75]):
        T, cu = sum(new), _ints(np.concatenate([[0], np.cumsum(new)]))
        cap = T + 5
        pos = np.concatenate([have[b] + np.arange(n) for b, n in enumerate(new)])
        rows = np.concatenate([[2 * table[b, j // page] * page + j % page for j in range(have[b], have[b] + n)]
                               for b, n in enumerate(new)]).astype(int)
        have = have + np.asarray(new)
        res = torch.randn((cap, C), generator=g).cuda()       # the residual stream in 32 bits
        x = torch.randn((cap, C), generator=g).to(BF).cuda()
        new_of = lambda *s, dt=BF: nan_fill(torch.empty(s, dtype=dt, device="cuda"))
        s1, s2, y1, y2 = new_of(cap, C, dt=torch.float32), new_of(cap, C, dt=torch.float32), new_of(cap, C, dt=E4), new_of(cap, C, dt=E4)
        a1, a2, qkv = new_of(cap, dt=torch.float32), new_of(cap, dt=torch.float32), new_of(cap, Hq + 2 * Hkv, d)
        qr, o, att, up = new_of(cap, Hq, d), new_of(cap, Hq, d), new_of(cap, C), new_of(cap, hidden)
        full = lambda v, fill: _ints(np.concatenate([v, np.full(cap - T, fill)]))
        rra.rms_norm(x, cu, 3, y1, weight=n1, residual=res, sum_out=s1, scale=a1)
        rra.linear_scaled(y1, a1, wqkv, sqkv, cu, 3, qkv.view(cap, -1))
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        # keys to rows `rows` of the pool, values to the rows of the other half of the same page
        rra.qk_norm_rope(q, k, full(pos, 0), cu, 3, qr, slots, inv_freq, q_weight=nq, k_weight=nk, kv_rows=full(rows, 0))
        slots[torch.as_tensor(rows + page, device="cuda")] = v[:T]
        rra.attend_paged(qr, kp, vp, _ints(table), _ints(have), cu, 3, max(new), int(have.max()), o, scale=d ** -0.5)
        rra.linear_epilogue(o.view(cap, -1), wo, cu, 3, att)
        rra.rms_norm(att, cu, 3, y2, weight=n2, residual=s1, sum_out=s2, scale=a2)
        rra.linear_scaled(y2, a2, wup, sup, cu, 3, up, act=rra.ACT_SILU)
        torch.cuda.synchronize()
        assert rra.get_device_error() == 0
        for xx, rr, ss, yy, aa, nn in ((x, res, s1, y1, a1, n1), (att, s1, s2, y2, a2, n2)):
            s64, y64 = OB.rms_norm(_np(xx)[:T], _np(rr)[:T], _np(nn), float(np.float32(1e-6)))
            sc = OB.row_scale(y64)
            assert np.all(np.abs(_np(ss)[:T] - s64) <= 2.0 ** -24 * np.abs(s64))
            assert np.all(np.abs(_np(aa)[:T] / sc - 1) <= 34 * 2.0 ** -24)
            v64, got = y64 / sc[:, None], _np(yy)[:T]
            e = np.abs(v64) * 67 * 2.0 ** -24
            assert np.all((OB.to_e4m3(v64 - e) <= got) & (got <= OB.to_e4m3(v64 + e)))
        for aa, sa, ww, sw, cc, act in ((y1, a1, wqkv, sqkv, qkv.view(cap, -1), "none"), (y2, a2, wup, sup, up, "silu")):
            a64, w64 = _np(aa)[:T] * _np(sa)[:T, None], _np(ww) * _np(sw)[:, None]
            ref, S = OB.linear_epilogue(a64, w64, None, act, None, T), np.abs(a64) @ np.abs(w64).T
            tol = 1.13 * F * (C + 1.5) * S + 16 * F * (1 + S)
            assert np.all(np.abs(_np(cc)[:T] - ref) <= tol + half_step(BF) * (np.abs(ref) + tol))
        at = 0
        for b, n in enumerate(new):
            m = int(have[b])
            kk, vv = (torch.from_numpy(OB.cached_rows(_np(t), table[b], m)) for t in (kp, vp))
            assert bool(torch.isfinite(kk).all() and torch.isfinite(vv).all())
            if n:
                check_rows(o[at:at + n].cpu(), qr[at:at + n].cpu(), kk, vv, d ** -0.5, m - n + np.arange(n), BF)
            at += n
        for t in (y1, y2, s1, s2, qkv, o, up):
            assert bool(torch.isnan(t[T:].float()).all())


def _step(seed, cap, T, dtype=BF):
    """A call of each operator on its own buffers, as a function, and the outputs it writes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)
    Hq, Hkv, d, C, page = 4, 2, 128, 336, 32
    x, res, w, b = r(cap, C), r(cap, C), (r(Hq * d, C, dt=torch.float32) * 40).to(E4), r(Hq * d, dt=torch.float32)
    sw = 0.01 * torch.rand(Hq * d, generator=g, device="cuda")
    sums, y, sc = torch.zeros_like(x), torch.zeros((cap, C), device="cuda").to(E4), torch.zeros(cap, device="cuda")
    q = torch.zeros((cap, Hq, d), dtype=dtype, device="cuda")
    pool = r(60, 2, page, Hkv, d)
    table = torch.randperm(60, generator=g, device="cuda").to(torch.int32).view(2, 30)
    n = [T // 3, T - T // 3]
    cu, lens = _ints([0, T // 3, T]), _ints([n[0] + 5, 900])
    o = torch.zeros_like(q)

    def call(stream=None, workspace=None):
        rra.rms_norm(x, cu, 2, y, residual=res, sum_out=sums, scale=sc, stream=stream)
        rra.linear_scaled(y, sc, w, sw, cu, 2, q.view(cap, -1), bias=b, act=rra.ACT_GELU_TANH, stream=stream)
        rra.attend_paged(q, pool[:, 0], pool[:, 1], table, lens, cu, 2, max(n), 900, o, scale=0.09, workspace=workspace,
                         stream=stream)

    return call, [sums, y, sc, q, o]


@pytest.mark.parametrize("cap,T", [(3, 3), (16, 9), (100, 77), (400, 391)])
def test_streams_graphs_and_calls_at_once(cap, T):
    """Eager, on another stream (given, and current), captured and replayed, and two at once: the same bits every time."""
    first, outs1 = _step(1, cap, T)
    second, outs2 = _step(2, cap, T)
    first(), second()
    torch.cuda.synchronize()
    bits = lambda x: x.view(torch.uint8)
    want = [x.clone() for x in outs1 + outs2]
    assert all(bool(torch.isfinite(x.float()).all()) for x in want)

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(want, outs1 + outs2))
        for x in outs1 + outs2:
            bits(x).zero_()
        torch.cuda.synchronize()

    for x in outs1 + outs2:
        bits(x).zero_()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        first(s1)
        with torch.cuda.stream(s2):
            second()
    check()
    graphs = []
    for call in (first, second):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append(gr)
    for _ in range(5):
        for gr, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                gr.replay()
    check()
    own = [rra.attend_paged_workspace(2, cap, max(T // 3, T - T // 3), 900, 4, 2, 128) for _ in range(2)]
    for _ in range(3):                                               # workspaces of the caller's, one a stream
        first(s1, own[0])
        second(s2, own[1])
    check()
    assert rra.get_device_error() == 0


def test_errors_go_to_the_bound_word():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    rra.get_device_error(clear=True)
    rra.bind_error_word(word)
    try:
        x = torch.zeros((4, 64), device="cuda")
        rra.rms_norm(x.half(), _ints([0, 5]), 1, x.half())
        assert rra.read_error_word(word) == rra.DEVERR_INDEX_RANGE
        one = torch.ones(64, device="cuda")
        rra.linear_scaled(x.to(E4), one[:4], torch.zeros((16, 64), device="cuda").to(E4), one[:16], _ints([0, 5]), 1,
                          torch.zeros((4, 16), device="cuda"))
        assert rra.read_error_word(word) == rra.DEVERR_INDEX_RANGE
        kv = torch.zeros((3, 16, 1, 64), device="cuda").half()
        for n in (1, 40):                                           # rows of a warp, tiles
            q = torch.zeros((n, 2, 64), device="cuda").half()
            rra.attend_paged(q, kv, kv.clone(), _ints([[0, 1, 2]]), _ints([49]), _ints([0, n]), 1, n, 48, q.clone(), scale=0.1)
            assert rra.read_error_word(word) == rra.DEVERR_SEQ_TOO_LONG
    finally:
        rra.bind_error_word(None)
    assert rra.get_device_error() == 0


def test_both_marshalling_paths_make_the_same_call(monkeypatch):
    """The C++ marshalling and the binding's own: the same bits, and the same refusals."""
    assert rra.lib() and rra._FAST is not None, "the marshalling extension was not built"
    call, outs = _step(5, 40, 37)
    call()
    torch.cuda.synchronize()
    bits = lambda x: x.view(torch.uint8)
    want = [x.clone() for x in outs]
    z = lambda *s, dt=BF: torch.zeros(s, device="cuda").to(dt)
    cu, f32 = _ints([0, 4]), torch.float32
    pool, table, one = z(3, 2, 16, 2, 64), _ints([[0, 1]]), _ints([4])
    k, v = pool[:, 0], pool[:, 1]
    bad = [
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 72)),                                               # y's shape
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 64), weight=z(64)),                                 # weight's type
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 64), residual=z(4, 64)),                            # no sum_out
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 64), residual=z(4, 64, dt=f32), sum_out=z(4, 64)),  # types differ
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 64, dt=E4)),                                        # no scale
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 64), scale=z(4, dt=f32)),                           # a scale too many
        lambda: rra.rms_norm(z(64, 4).t(), cu, 1, z(4, 64)),                                           # not contiguous
        lambda: rra.rms_norm(z(4, 60), cu, 1, z(4, 60)),                                               # the library's own
        lambda: rra.rms_norm(z(4, 64), cu, 1, z(4, 64, dt=f32)),
        lambda: rra.linear_scaled(z(4, 64, dt=E4), z(4, dt=f32), z(8, 64), z(8, dt=f32), cu, 1, z(4, 8)),
        lambda: rra.linear_scaled(z(4, 64, dt=E4), z(5, dt=f32), z(8, 64, dt=E4), z(8, dt=f32), cu, 1, z(4, 8)),
        lambda: rra.linear_scaled(z(4, 64, dt=E4), z(4, dt=f32), z(8, 64, dt=E4), z(8), cu, 1, z(4, 8)),
        lambda: rra.linear_scaled(z(4, 72, dt=E4), z(4, dt=f32), z(8, 72, dt=E4), z(8, dt=f32), cu, 1, z(4, 8)),
        lambda: rra.attend_paged(z(4, 2, 64), k, z(3, 16, 2, 64), table, one, cu, 1, 4, 32, z(4, 2, 64), scale=0.1),
        lambda: rra.attend_paged(z(4, 2, 64), k, v, table, one, cu, 2, 4, 32, z(4, 2, 64), scale=0.1),
        lambda: rra.attend_paged(z(4, 2, 64), k, v, table.long(), one, cu, 1, 4, 32, z(4, 2, 64), scale=0.1),
        lambda: rra.attend_paged(z(4, 2, 64), k, v, table, one, cu, 1, 4, 32, z(4, 1, 64), scale=0.1),
        lambda: rra.attend_paged(z(4, 2, 64), pool[:, 0].transpose(1, 2), v, table, one, cu, 1, 4, 32, z(4, 2, 64), scale=0.1),
        lambda: rra.attend_paged(z(4, 2, 64), k, v, table, one, cu, 1, 4, 33, z(4, 2, 64), scale=0.1),  # the library's own
        lambda: rra.attend_paged(z(24, 2, 64), k, v, table, one, cu, 1, 24, 32, z(24, 2, 64), scale=0.1, workspace=z(16, dt=torch.uint8)),
    ]
    kinds = []
    for f in bad:
        with pytest.raises((ValueError, rra.RRAError)) as e:
            f()
        kinds.append((type(e.value), getattr(e.value, "status", None)))
    monkeypatch.setattr(rra, "_FAST", None)
    for x in outs:
        bits(x).zero_()
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(want, outs))
    for f, kind in zip(bad, kinds):
        with pytest.raises((ValueError, rra.RRAError)) as e:
            f()
        assert (type(e.value), getattr(e.value, "status", None)) == kind


def test_first_calls_may_be_captured():
    """In a fresh process, the first call of every operator inside a stream capture, replayed against the eager result."""
    code = """
import torch
from ragged_attention_token_gb300 import rra
g = torch.Generator(device="cuda").manual_seed(1)
e4 = torch.float8_e4m3fn
r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
caps = (8, 100, 300)
x, w, ones = [r(n, 256) for n in caps], r(128, 256).to(e4), torch.ones(512, device="cuda")
cus = [ints([0, n]) for n in caps]
y, y16 = [torch.zeros(n, 256, device="cuda").to(e4) for n in caps], [torch.zeros_like(a) for a in x]
sc = [torch.zeros(n, device="cuda") for n in caps]
c = [torch.zeros(n, 128, device="cuda").bfloat16() for n in caps]
pool, table = r(40, 2, 32, 2, 64), torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
qs = [r(n, 4, 64) for n in (1, 300)]
os_ = [torch.zeros_like(q) for q in qs]
cuq = [ints([0, 1]), ints([0, 300])]
lens = ints([1000])
def step():
    for i in range(3):
        rra.rms_norm(x[i], cus[i], 1, y[i], scale=sc[i])
        rra.rms_norm(x[i], cus[i], 1, y16[i])
        rra.linear_scaled(y[i], sc[i], w, ones[:128], cus[i], 1, c[i])
    for i, n in enumerate((1, 300)):
        rra.attend_paged(qs[i], pool[:, 0], pool[:, 1], table, lens, cuq[i], 1, n, 1000, os_[i], scale=0.1)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    step()
gr.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (*y16, *c, *os_)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (*y16, *c, *os_))) and bool(got[-1].float().abs().sum() > 0)
assert rra.get_device_error() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and "captured" in out.stdout, out.stdout + out.stderr


def _linear(cap, K, N, out):
    g = torch.Generator(device="cuda").manual_seed(cap + K + N)
    a, w = ((torch.randn(s, generator=g, device="cuda") * 60).to(E4) for s in ((cap, K), (N, K)))
    one = torch.ones(max(cap, N), device="cuda")
    c = torch.empty((cap, N), dtype=out, device="cuda")
    cu = _ints([0, cap])
    return c, lambda: rra.linear_scaled(a, one[:cap], w, one[:N], cu, 1, c)


def _paged(new, kv, Hq, Hkv, d, dtype=BF, page=32):
    g = torch.Generator(device="cuda").manual_seed(sum(kv))
    need = -(-max(kv) // page)
    pool = torch.randn((need * len(kv), 2, page, Hkv, d), generator=g, device="cuda").to(dtype)
    table = torch.randperm(need * len(kv), generator=g, device="cuda").to(torch.int32).view(len(kv), need)
    q = torch.randn((sum(new), Hq, d), generator=g, device="cuda").to(dtype)
    o, cu, lens = torch.empty_like(q), _ints(np.concatenate([[0], np.cumsum(new)])), _ints(kv)
    return o, lambda: rra.attend_paged(q, pool[:, 0], pool[:, 1], table, lens, cu, len(kv), max(new), max(kv), o, scale=d ** -0.5)


LIMITED = {
    "mid": lambda: _linear(64, 8192, 4096, BF),
    "pair": lambda: _linear(3000, 2048, 2304, BF),
    "pair_parts": lambda: _linear(3000, 8192, 2304, torch.float32),
    "paged_chunk": lambda: _paged([2000, 100], [4000, 100], 16, 4, 128),
    "paged_tokens": lambda: _paged([3] * 9, [5000, 100, 1, 17, 9000, 3, 5, 4000, 1000], 16, 2, 64, torch.float16),
    "paged_one": lambda: _paged([60], [60000], 2, 1, 128),
}


def _under(call, cycles):
    rra.get_device_error(clear=True)
    old = rra.set_wait_limit(cycles)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        rra.set_wait_limit(old)
    return rra.get_device_error(clear=True)


@pytest.mark.parametrize("name", list(LIMITED))
def test_waits_that_run_out(name):
    """With a limit that runs out the call says so and returns, what it wrote is right or as it was, and the next normal
    call is right."""
    out, call = LIMITED[name]()
    out.fill_(float("nan"))
    rra.get_device_error(clear=True)
    call()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    want = out.clone()
    assert bool(torch.isfinite(want.float()).all())
    assert _under(call, 100) == rra.DEVERR_WAIT_TIMEOUT
    out.fill_(float("nan"))
    assert _under(call, 10 ** 10) == 0
    assert torch.equal(out, want)
    for cycles in (400, 700, 1000, 1500, 2000, 3000, 4000, 6000, 8000, 12000, 20000):
        out.fill_(float("nan"))
        _under(call, cycles)
        assert bool(((out == want) | torch.isnan(out)).all()), cycles
    out.fill_(float("nan"))
    call()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("m", [399992, 400000])
@pytest.mark.parametrize("d", [64, 128])
def test_a_long_piece_is_no_long_wait(m, d):
    """The bound is for one wait of a block: pieces whose walk takes longer than it pass, whether the last block ends in
    a tail or not."""
    out, call = _paged([33, 64], [m, m - 7], 64, 32, d, page=64) if d == 64 else _paged([33], [m], 64, 32, d, page=64)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    assert bool(torch.isfinite(want.float()).all())
    out.fill_(float("nan"))
    assert _under(call, 300000) == 0
    assert torch.equal(out, want)
