"""Refusals of the row norm, the 8-bit linear layer and the attention over pages, at the C ABI and in the binding (CPU:
every check precedes any CUDA call)."""
import numpy as np
import pytest
import torch

from oracle import block as OB
from ragged_attention_token_gb300 import build, rra

INV, UNS, MIS = rra.RRA_ERR_INVALID_ARG, rra.RRA_ERR_UNSUPPORTED, rra.RRA_ERR_MISALIGNED
NAN = float("nan")
BF, F32, E4 = rra.RRA_BF16, rra.RRA_F32, rra.RRA_E4M3


@pytest.fixture(scope="module")
def L():
    if not build.up_to_date():
        build.build()
    return rra.lib()


def _call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return fn(*a.values())


NORM = dict(x=0x1000000, res=0x2000000, rdt=BF, w=0x100, eps=1e-6, cu=0x8000, B=1, cap=512, N=384, dt=BF, sum=0x3000000,
            y=0x4000000, out=E4, scale=0x9000, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=380), UNS), (dict(N=0), UNS), (dict(N=32776), UNS), (dict(B=0), INV), (dict(B=65536), INV), (dict(cap=0), INV),
    (dict(dt=F32), INV), (dict(dt=E4), INV), (dict(out=F32, scale=None), INV), (dict(out=rra.RRA_F16, scale=None), INV),
    (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=float("inf")), INV), (dict(rdt=rra.RRA_F16), INV),
    (dict(rdt=E4), INV), (dict(sum=None), INV), (dict(res=None), INV), (dict(scale=None), INV), (dict(out=BF), INV),
    (dict(x=None), INV), (dict(y=None), INV), (dict(cu=None), INV), (dict(cu=0x8002), MIS), (dict(x=0x1000008), MIS),
    (dict(res=0x2000004), MIS), (dict(sum=0x3000008), MIS), (dict(y=0x4000008), MIS), (dict(w=0x104), MIS),
    (dict(scale=0x9002), MIS), (dict(y=0x1000000), INV),                     # 8 bits over x
    (dict(y=0x1000010, out=BF, scale=None), INV),                            # over x, shifted
    (dict(y=0x3000000), INV), (dict(y=0x2000000, out=BF, scale=None), INV),  # over the sum, over the residual
    (dict(sum=0x2000010), INV), (dict(sum=0x1000000, rdt=F32), INV),         # 32 bits over x
    (dict(sum=0x100), INV), (dict(y=0x100 + 16), INV), (dict(scale=0x1000000), INV), (dict(scale=0x4000000), INV),
    (dict(scale=0x3000000), INV), (dict(scale=0x2000000), INV), (dict(scale=0x104), INV)])
def test_rms_norm_refusals(L, kw, want):
    assert _call(L.rra_rms_norm, NORM, kw) == want


LIN = dict(a=0x1000000, sa=0x8000, w=0x2000000, sw=0x9000, bias=0x100, res=None, cu=0x300, B=1, cap=512, K=384, N=1152,
           act=0, c=0x4000000, out=BF, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=392), UNS), (dict(K=0), UNS), (dict(K=65552), UNS), (dict(N=100), UNS), (dict(N=0), UNS), (dict(B=0), INV),
    (dict(cap=0), INV), (dict(cap=65535 * 128 + 1), INV), (dict(out=E4), INV), (dict(act=5), INV), (dict(act=-1), INV),
    (dict(a=None), INV), (dict(w=None), INV), (dict(c=None), INV), (dict(cu=None), INV), (dict(sa=None), INV),
    (dict(sw=None), INV), (dict(cu=0x302), MIS), (dict(a=0x1000008), MIS), (dict(sa=0x8002), MIS), (dict(sw=0x9008), MIS),
    (dict(bias=0x104), MIS), (dict(res=0x5000008), MIS), (dict(c=0x1000000), INV),
    (dict(c=0x1000000 + 512 * 384 - 16), INV), (dict(c=0x2000000), INV), (dict(bias=0x4000000), INV),
    (dict(sa=0x4000000), INV), (dict(sw=0x4000010), INV), (dict(res=0x4000010), INV)])
def test_linear_scaled_refusals(L, kw, want):
    assert _call(L.rra_linear_scaled, LIN, kw) == want


PAGED = dict(q=0x1000000, qs=2048, k=0x20000000, v=0x30000000, ps=64 * 2 * 128, pages=9, page=64, table=0x400, width=4,
             lens=0x300, cu=0x500, B=2, cap=64, new=64, kv=256, Hq=16, Hkv=2, d=128, scale=0.1, dt=rra.RRA_F16, o=0x4000000,
             ws=0x50000000, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=256), UNS), (dict(page=8), UNS), (dict(page=24), UNS), (dict(page=0), UNS), (dict(page=65552), UNS),
    (dict(pages=0), INV), (dict(width=0), INV), (dict(new=0), INV), (dict(new=(1 << 30) + 1), UNS), (dict(kv=0), INV),
    (dict(kv=257), INV), (dict(kv=(1 << 30) + 1, width=1 << 30), UNS), (dict(B=0), INV), (dict(cap=0), INV),
    (dict(Hq=5), INV), (dict(scale=NAN), INV), (dict(scale=-0.5), INV), (dict(dt=F32), INV), (dict(dt=E4), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(lens=None), INV), (dict(cu=None), INV),
    (dict(table=None), INV), (dict(o=None), INV), (dict(lens=0x301), MIS), (dict(table=0x402), MIS), (dict(cu=0x501), MIS),
    (dict(k=0x20000004), MIS), (dict(v=0x30000008), MIS), (dict(qs=2052), MIS), (dict(qs=2040), INV),
    (dict(ps=64 * 2 * 128 - 8), INV), (dict(ps=64 * 2 * 128 + 4), MIS), (dict(ps=1 << 36), INV), (dict(o=0x20000000), INV),
    (dict(o=0x30000000 + 9 * 64 * 2 * 128 * 2 - 16), INV), (dict(o=0x1000000 + 2048), INV), (dict(ws=None), INV),
    (dict(wsb=1000), INV), (dict(ws=0x50000010), MIS), (dict(ws=0x4000000 - 256), INV), (dict(ws=0x1000000), INV),
    (dict(Hq=4000, Hkv=1, qs=4000 * 128, B=65535, cap=1 << 20, new=1 << 20), UNS), (dict(ws=0x20000100), INV), (dict(ws=0x30000000 - 256), INV)])
def test_attend_paged_refusals(L, kw, want):
    assert _call(L.rra_attend_paged, PAGED, kw) == want


def test_attend_paged_workspace_bytes(L):
    f = lambda B=2, cap=64, new=64, kv=256, Hq=16, Hkv=2, d=128: L.rra_attend_paged_workspace_bytes(B, cap, new, kv, Hq, Hkv, d)
    assert f(new=1) == 0 and f(new=2) == 0                                  # a few rows on short caches need none
    assert 0 < f(new=1, kv=1 << 20) <= f(new=3) < f(new=6) < f() == f(new=1 << 30)
    assert f(cap=1) == 0                                                    # no more new tokens than rows
    assert f(Hq=256, Hkv=1, d=64) == 0                                      # more heads to a group than a tile has rows
    assert f(new=0) == 0 and f(kv=0) == 0 and f(B=0) == 0 and f(Hkv=3) == 0 and f(d=96) == 0


def test_binding_refuses_before_the_library():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    cu, f32, e4 = torch.zeros(2, dtype=torch.int32), torch.float32, torch.float8_e4m3fn
    with pytest.raises(ValueError):                                         # host tensors
        rra.rms_norm(z(4, 64), cu, 1, z(4, 64))
    with pytest.raises(ValueError):                                         # residual without sum_out
        rra.rms_norm(z(4, 64), cu, 1, z(4, 64), residual=z(4, 64))
    with pytest.raises(ValueError):                                         # 8 bits without scale
        rra.rms_norm(z(4, 64), cu, 1, z(4, 64, dt=e4))
    with pytest.raises(ValueError):                                         # scale without 8 bits
        rra.rms_norm(z(4, 64), cu, 1, z(4, 64), scale=z(4, dt=f32))
    with pytest.raises(ValueError):                                         # 16-bit weights of the layer
        rra.linear_scaled(z(4, 64, dt=e4), z(4, dt=f32), z(8, 64), z(8, dt=f32), cu, 1, z(4, 8))
    pool = z(3, 2, 16, 2, 64)
    table = torch.zeros((1, 2), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):                                         # host tensors
        rra.attend_paged(z(4, 2, 64), pool[:, 0], pool[:, 1], table, one, cu, 1, 4, 32, z(4, 2, 64), scale=0.125)
    with pytest.raises(ValueError):                                         # pages of another stride
        rra.attend_paged(z(4, 2, 64), pool[:, 0], z(3, 16, 2, 64), table, one, cu, 1, 4, 32, z(4, 2, 64), scale=0.125)


def test_oracle_rounds_to_8_bits_as_torch_does():
    """The oracle's e4m3 against torch's conversion: every value, the middle of every two neighbours and what lies beside it."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = torch.unique(every[torch.isfinite(every)]).double()
    mid = (every[1:] + every[:-1]) / 2
    v = torch.cat([every, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)]).float()
    assert np.array_equal(OB.to_e4m3(v.double().numpy()), v.to(torch.float8_e4m3fn).double().numpy())


def test_no_read_only_loads_in_programmatic_dependents():
    """As for the block's other kernels: what starts before the kernels ahead of it have finished reads by ordinary loads."""
    import os
    import re
    seen = set()
    for f in os.listdir(build.CSRC):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, f)).read())
        if "start_dependent();" in text:
            seen.add(f)
            assert "__ldg" not in text and "ld.global.nc" not in text and "__restrict__" not in text, f
    assert {"rms_norm.cu", "attend_paged.cu"} <= seen
