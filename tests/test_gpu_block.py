"""The block operators together, as a model uses them (needs a GPU): a layer's attention half over packed prompts
(projection, norm and rotation in place, attention, projection onto the residual) with its keys and values written into
a cache, then one more token of every sequence against that cache.  The oracle computes both in fp64 from the
same weights; the one-token step must agree with the prompt pass over the longer prompts."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(8, 2, 128, torch.bfloat16), (6, 6, 64, torch.float16)])
def test_prompt_then_one_token(Hq, Hkv, d, dtype):
    g = torch.Generator().manual_seed(11)
    C, lens = 384, [150, 1, 33]
    full = [n + 1 for n in lens]                                     # prompts with the next token appended
    B, cap_kv, W = len(lens), 200, (Hq + 2 * Hkv) * d
    w1 = (torch.randn((W, C), generator=g) / np.sqrt(C)).to(dtype)
    w2 = (torch.randn((C, Hq * d), generator=g) / np.sqrt(Hq * d)).to(dtype)
    b1 = 0.1 * torch.randn(W, generator=g)
    nw = 1 + 0.1 * torch.randn((2, d), generator=g)
    f = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float()
    x_full = torch.randn((sum(full), C), generator=g).to(dtype)
    w1d, w2d, b1d, nwd, fd = w1.cuda(), w2.cuda(), b1.cuda(), nw.cuda(), f.cuda()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def layer(x, lens, attend, positions, slots, kc, vc):
        T = x.shape[0]
        cu = ints(np.concatenate([[0], np.cumsum(lens)]))
        qkv = torch.empty((T, Hq + 2 * Hkv, d), dtype=dtype, device="cuda")
        rra.linear_epilogue(x, w1d, cu, len(lens), qkv.view(T, W), bias=b1d)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if slots is not None:
            rra.qk_norm_rope(q, k, positions, cu, len(lens), q, kc, fd, q_weight=nwd[0], k_weight=nwd[1], v=v, v_out=vc,
                             kv_rows=slots)
        if slots is None or attend == "prompt":
            rra.qk_norm_rope(q, k, positions, cu, len(lens), q.clone() if slots is not None else q, k, fd,
                             q_weight=nwd[0], k_weight=nwd[1])
        o = torch.empty((T, Hq, d), dtype=dtype, device="cuda")
        if attend == "prompt":
            rra.attend_prompt(q, k, v, cu, len(lens), max(lens), o, scale=d ** -0.5)
        else:
            rra.attend_cache(q, kc.view(B, cap_kv, Hkv, d), vc.view(B, cap_kv, Hkv, d), attend, o, scale=d ** -0.5)
        y = x.clone()
        rra.linear_epilogue(o.view(T, Hq * d), w2d, cu, len(lens), y, residual=y)
        return y

    kc, vc = (torch.zeros((B * cap_kv, Hkv, d), dtype=dtype, device="cuda") for _ in range(2))
    at = np.concatenate([[0], np.cumsum(full)])
    prompt_rows = np.concatenate([np.arange(at[b], at[b] + lens[b]) for b in range(B)])
    last_rows = at[1:] - 1
    pos = ints(np.concatenate([np.arange(n) for n in lens]))
    slots = ints(np.concatenate([b * cap_kv + np.arange(n) for b, n in enumerate(lens)]))
    rra.get_device_error(clear=True)
    y_prompt = layer(x_full[prompt_rows].cuda(), lens, "prompt", pos, slots, kc, vc)
    y_next = layer(x_full[last_rows].cuda(), [1] * B, ints([n + 1 for n in lens]), ints(lens),
                   ints([b * cap_kv + n for b, n in enumerate(lens)]), kc, vc)
    y_full = layer(x_full.cuda(), full, "prompt", ints(np.concatenate([np.arange(n) for n in full])), None, None, None)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0

    x64 = x_full.double().numpy()
    qkv = OB.linear_epilogue(x64, w1.double().numpy(), b1.double().numpy(), "none", None, len(x64)).reshape(-1, Hq + 2 * Hkv, d)
    p64 = np.concatenate([np.arange(n) for n in full])
    f64, n64 = f.double().numpy(), nw.double().numpy()
    q = OB.norm_rope(qkv[:, :Hq], p64, n64[0], 1e-6, f64, False, 1.0)
    k = OB.norm_rope(qkv[:, Hq:Hq + Hkv], p64, n64[1], 1e-6, f64, False, 1.0)
    o = np.concatenate([OB.attend_rows(q[at[b]:at[b + 1]], k[at[b]:at[b + 1]], qkv[at[b]:at[b + 1], Hq + Hkv:], d ** -0.5,
                                       np.arange(full[b]))[0] for b in range(B)])
    y = OB.linear_epilogue(o.reshape(-1, Hq * d), w2.double().numpy(), None, "none", x64, len(x64))
    # Four roundings to the type on the way (projection, norm/rotation, weights and output of the attention), each at
    # most half a step of values of order one to five, through sums whose weights' squares add up to one, and the last
    # rounding: within 24 half steps of 1 + |y|.
    u = torch.finfo(dtype).eps / 2
    for got, rows in ((y_prompt, prompt_rows), (y_next, last_rows), (y_full, np.arange(len(x64)))):
        err = np.abs(got.cpu().double().numpy() - y[rows])
        assert np.all(err <= 24 * u * (1 + np.abs(y[rows]))), float(err.max())


def _step(seed, cap, T, dtype=torch.bfloat16):
    """A call of each operator on its own buffers, as a function, and the outputs it writes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(s, generator=g, device="cuda").to(dt)
    Hq, Hkv, d, C, R = 4, 2, 128, 320, 700
    x, w, b = r(cap, C), r((Hq + 2 * Hkv) * d, C), r((Hq + 2 * Hkv) * d, dt=torch.float32)
    res = r(cap, (Hq + 2 * Hkv) * d)
    qkv = torch.zeros((cap, Hq + 2 * Hkv, d), dtype=dtype, device="cuda")
    qo, ko = torch.zeros((cap, Hq, d), dtype=dtype, device="cuda"), torch.zeros((cap, Hkv, d), dtype=dtype, device="cuda")
    o, oc = torch.zeros_like(qo), torch.zeros((2, Hq, d), dtype=dtype, device="cuda")
    kc, vc = r(2, R, Hkv, d), r(2, R, Hkv, d)
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    pos = torch.arange(cap, dtype=torch.int32, device="cuda")
    f = 10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))
    lens = torch.tensor([R, 33], dtype=torch.int32, device="cuda")

    def call(stream=None):
        rra.linear_epilogue(x, w, cu, 2, qkv.view(cap, -1), bias=b, act=rra.ACT_SILU, residual=res, stream=stream)
        rra.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], pos, cu, 2, qo, ko, f, q_weight=f.new_ones(d), stream=stream)
        rra.attend_prompt(qo, ko, qkv[:, Hq + Hkv:], cu, 2, T, o, scale=0.09, stream=stream)
        rra.attend_cache(qo[:2], kc, vc, lens, oc, scale=0.09, stream=stream)

    return call, [qkv, qo, ko, o, oc]


@pytest.mark.parametrize("cap,T", [(3, 3), (16, 9), (100, 77), (400, 391)])
def test_streams_graphs_and_calls_at_once(cap, T):
    """Eager, on another stream (given, and current), captured and replayed, and two at once: the same bits every time."""
    first, outs1 = _step(1, cap, T)
    second, outs2 = _step(2, cap, T)
    first(), second()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs1 + outs2]
    assert all(bool(torch.isfinite(x.float()).all()) for x in want)

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs1 + outs2))
        for x in outs1 + outs2:
            x.zero_()
        torch.cuda.synchronize()

    for x in outs1 + outs2:
        x.zero_()
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
    assert rra.get_device_error() == 0


def test_errors_go_to_the_bound_word():
    """A thread's bound error word takes the block operators' codes too, and the device's own word stays clear."""
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    rra.get_device_error(clear=True)
    rra.bind_error_word(word)
    try:
        a, w = torch.zeros((4, 64), device="cuda").bfloat16(), torch.zeros((16, 64), device="cuda").bfloat16()
        c = torch.zeros((4, 16), device="cuda")
        rra.linear_epilogue(a, w, torch.tensor([0, 5], dtype=torch.int32, device="cuda"), 1, c)
        assert rra.read_error_word(word) == rra.DEVERR_INDEX_RANGE
        x = torch.zeros((2, 1, 64), device="cuda").half()
        rra.attend_prompt(x, x.clone(), x.clone(), torch.tensor([0, 2], dtype=torch.int32, device="cuda"), 1, 1,
                          x.clone(), scale=0.1)
        assert rra.read_error_word(word) == rra.DEVERR_SEQ_TOO_LONG
        kv = torch.zeros((2, 3, 1, 64), device="cuda").half()
        rra.attend_cache(x, kv, kv.clone(), torch.tensor([4, 1], dtype=torch.int32, device="cuda"), x.clone(), scale=0.1)
        assert rra.read_error_word(word) == rra.DEVERR_SEQ_TOO_LONG
        rra.qk_norm_rope(x, x.clone(), None, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 1, x.clone(), x.clone())
        assert rra.read_error_word(word) == rra.DEVERR_INDEX_RANGE
    finally:
        rra.bind_error_word(None)
    assert rra.get_device_error() == 0


def test_both_marshalling_paths_make_the_same_call(monkeypatch):
    """The C++ marshalling and the binding's own: the same bits, and the same refusals."""
    assert rra.lib() and rra._FAST is not None, "the marshalling extension was not built"
    call, outs = _step(5, 40, 37)
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bad = [
        lambda: rra.linear_epilogue(z(4, 64), z(8, 72), cu, 1, z(4, 8)),                               # K differs
        lambda: rra.linear_epilogue(z(4, 64), z(8, 64), cu, 1, z(4, 8), bias=z(8)),                    # bias type
        lambda: rra.linear_epilogue(z(64, 4).t(), z(8, 64), cu, 1, z(4, 8)),                           # not contiguous
        lambda: rra.linear_epilogue(z(4, 64), z(8, 64), cu, 2, z(4, 8)),                               # cu too short
        lambda: rra.linear_epilogue(z(4, 64), z(8, 64), cu.long(), 1, z(4, 8)),                        # cu type
        lambda: rra.attend_prompt(z(4, 2, 64), z(4, 2, 64), z(4, 1, 64), cu, 1, 4, z(4, 2, 64), scale=0.1),
        lambda: rra.attend_prompt(z(4, 64, 2).transpose(1, 2), z(4, 2, 64), z(4, 2, 64), cu, 1, 4, z(4, 2, 64), scale=0.1),
        lambda: rra.attend_cache(z(3, 2, 64), z(2, 8, 2, 64), z(2, 8, 2, 64), cu, z(3, 2, 64), scale=0.1),
        lambda: rra.qk_norm_rope(z(4, 2, 64), z(4, 2, 64), None, cu, 1, z(4, 2, 64), z(4, 2, 64).cpu()),
        lambda: rra.qk_norm_rope(z(4, 2, 64), z(4, 2, 64), None, cu, 1, z(4, 2, 64), z(4, 2, 64), v=z(4, 2, 64)),
        lambda: rra.linear_epilogue(z(4, 60), z(8, 60), cu, 1, z(4, 8)),                               # the library's own
        lambda: rra.attend_prompt(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), cu, 1, 4, z(4, 2, 64), scale=-0.1),
    ]
    kinds = []
    for f in bad:
        with pytest.raises((ValueError, rra.RRAError)) as e:
            f()
        kinds.append((type(e.value), getattr(e.value, "status", None)))
    monkeypatch.setattr(rra, "_FAST", None)
    for x in outs:
        x.zero_()
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    for f, kind in zip(bad, kinds):
        with pytest.raises((ValueError, rra.RRAError)) as e:
            f()
        assert (type(e.value), getattr(e.value, "status", None)) == kind


def test_first_calls_may_be_captured():
    """In a fresh process, the first call of every operator inside a stream capture (kernels and the rest of a
    device's set-up load there), replayed against the eager result."""
    code = """
import torch
from ragged_attention_token_gb300 import rra
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
x, w, q, kc = r(300, 64), r(128, 64), r(300, 4, 128), r(2, 700, 2, 128)
cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
ln = torch.tensor([700, 5], dtype=torch.int32, device="cuda")
c = [torch.zeros(n, 128, device="cuda").bfloat16() for n in (8, 100, 300)]
qo, ko, o, oc = (torch.zeros_like(y) for y in (q, q[:, :2], q, q[:2]))
cus = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (8, 100, 300)]
ones = torch.ones(128, device="cuda")
k2 = q[:, 2:].contiguous()
x8, x100 = x[:8].contiguous(), x[:100].contiguous()
q2 = q[:2].contiguous()
def step():
    for a, n, y in zip((x8, x100, x), cus, c):
        rra.linear_epilogue(a, w, n, 1, y)
    rra.qk_norm_rope(q, k2, None, cu, 1, qo, ko, q_weight=ones)
    rra.attend_prompt(q, k2, k2, cu, 1, 300, o, scale=0.1)
    rra.attend_cache(q2, kc, kc, ln, oc, scale=0.1)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    step()
gr.replay()
torch.cuda.synchronize()
got = [y.clone() for y in (*c, qo, ko, o, oc)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (*c, qo, ko, o, oc))) and bool(got[-1].float().abs().sum() > 0)
assert rra.get_device_error() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and "captured" in out.stdout, out.stdout + out.stderr
