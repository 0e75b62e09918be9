"""Refusals of the block operators, at the C ABI and in the binding (CPU: every check precedes any CUDA call)."""
import pytest
import torch

from ragged_attention_token_gb300 import build, rra

OK, INV, UNS, MIS = rra.RRA_OK, rra.RRA_ERR_INVALID_ARG, rra.RRA_ERR_UNSUPPORTED, rra.RRA_ERR_MISALIGNED
NAN = float("nan")


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


LIN = dict(a=0x1000000, w=0x2000000, bias=0x100, residual=None, cu=0x300, B=1, cap=512, K=384, N=1152,
           ind=rra.RRA_BF16, act=0, c=0x4000000, outd=rra.RRA_BF16, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=388), UNS), (dict(K=0), UNS), (dict(K=65544), UNS), (dict(N=100), UNS), (dict(N=0), UNS),
    (dict(B=0), INV), (dict(cap=0), INV), (dict(cap=65535 * 128 + 1), INV), (dict(ind=rra.RRA_F32), INV),
    (dict(outd=3), INV), (dict(act=5), INV), (dict(act=-1), INV), (dict(a=None), INV), (dict(w=None), INV),
    (dict(c=None), INV), (dict(cu=None), INV), (dict(cu=0x302), MIS), (dict(a=0x1000008), MIS),
    (dict(bias=0x104), MIS), (dict(residual=0x5000008), MIS), (dict(c=0x1000000), INV),
    (dict(c=0x1000000 + 512 * 384 * 2 - 16), INV), (dict(c=0x2000000 - 16), INV), (dict(bias=0x4000000), INV),
    (dict(residual=0x4000000 + 16), INV)])
def test_linear_epilogue_refusals(L, kw, want):
    assert _call(L.rra_linear_epilogue, LIN, kw) == want


ROPE = dict(q=0x1000000, qs=2560, k=0x1000000 + 2048 * 2, ks=2560, v=0x1000000 + 2304 * 2, vs=2560, pos=0x100, cu=0x300,
            B=2, cap=64, Hq=16, Hkv=2, d=128, dt=rra.RRA_BF16, qw=0x2000, kw=0x3000, eps=1e-6, f=0x4000, rot=128, il=0,
            rs=1.0, qo=0x2000000, qos=2048, ko=0x3000000, kos=256, vo=0x4000000, vos=256, rows=None, orows=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=96), UNS), (dict(rot=24), UNS), (dict(rot=144), UNS), (dict(rot=-16), UNS), (dict(Hq=15), INV),
    (dict(Hkv=0), INV), (dict(B=0), INV), (dict(cap=0), INV), (dict(dt=rra.RRA_F32), INV), (dict(eps=-1.0), INV),
    (dict(eps=NAN), INV), (dict(rs=float("inf")), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(qo=None), INV),
    (dict(ko=None), INV), (dict(v=None), INV), (dict(vo=None), INV), (dict(pos=None), INV), (dict(f=None), INV),
    (dict(cu=None), INV), (dict(cu=0x301), MIS), (dict(pos=0x102), MIS), (dict(rows=0x202, orows=64), MIS),
    (dict(rows=0x200, orows=0), INV), (dict(qs=2044), INV), (dict(qs=2564), MIS), (dict(ks=255), INV),
    (dict(q=0x1000008), MIS), (dict(qw=0x2004), MIS),
    (dict(qo=0x1000000, qos=2048), INV),                                   # over q, another stride
    (dict(qo=0x1000000 + 16, qos=2560), INV),                              # over q, shifted
    (dict(ko=0x1000000 + 2048 * 2, kos=2560, rows=0x200, orows=64), INV),  # k in place, but by slots
    (dict(ko=0x2000000), INV), (dict(vo=0x3000000), INV),                  # two outputs together
    (dict(qo=0x1000000 + 256 * 2, qos=2560), INV)])
def test_qk_norm_rope_refusals(L, kw, want):
    assert _call(L.rra_qk_norm_rope, ROPE, kw) == want


PROMPT = dict(q=0x1000000, qs=2560, k=0x1000000 + 2048 * 2, ks=2560, v=0x1000000 + 2304 * 2, vs=2560, cu=0x300, B=2,
              cap=64, S=64, Hq=16, Hkv=2, d=128, scale=0.1, causal=1, dt=rra.RRA_BF16, o=0x2000000, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=32), UNS), (dict(S=0), INV), (dict(S=(1 << 30) + 1), UNS), (dict(Hq=3), INV), (dict(B=0), INV),
    (dict(cap=0), INV), (dict(scale=NAN), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("inf")), INV), (dict(dt=rra.RRA_F32), INV), (dict(q=None), INV), (dict(o=None), INV),
    (dict(cu=None), INV), (dict(cu=0x302), MIS), (dict(v=0x1000008), MIS), (dict(ks=2556), MIS), (dict(vs=128), INV),
    (dict(o=0x1000000), INV), (dict(o=0x1000000 + 64 * 2560 * 2 - 640), INV)])
def test_attend_prompt_refusals(L, kw, want):
    assert _call(L.rra_attend_prompt, PROMPT, kw) == want


CACHE = dict(q=0x1000000, qs=2048, k=0x2000000, v=0x3000000, lens=0x300, B=2, nq=1, cap=64, Hq=16, Hkv=2, d=128,
             scale=0.1, dt=rra.RRA_F16, o=0x4000000, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=256), UNS), (dict(nq=0), UNS), (dict(nq=65), UNS), (dict(B=65535, Hkv=4096, Hq=4096, qs=4096 * 128), UNS), (dict(B=0), INV), (dict(cap=0), INV), (dict(Hq=5), INV),
    (dict(scale=NAN), INV), (dict(scale=-0.5), INV), (dict(dt=rra.RRA_F32), INV), (dict(q=None), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(lens=None), INV), (dict(o=None), INV), (dict(lens=0x301), MIS),
    (dict(k=0x2000004), MIS), (dict(qs=2052), MIS), (dict(qs=2040), INV), (dict(o=0x2000000), INV),
    (dict(o=0x1000000 + 2048), INV)])
def test_attend_cache_refusals(L, kw, want):
    assert _call(L.rra_attend_cache, CACHE, kw) == want


def test_binding_refuses_before_the_library():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):                                         # host tensors
        rra.attend_prompt(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), cu, 1, 4, z(4, 2, 64), scale=0.125)
    with pytest.raises(ValueError):                                         # v of another type
        rra.attend_prompt(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64, dt=torch.float16), cu, 1, 4, z(4, 2, 64), scale=0.125)
    with pytest.raises(ValueError):                                         # v without v_out
        rra.qk_norm_rope(z(4, 2, 64), z(4, 2, 64), None, cu, 1, z(4, 2, 64), z(4, 2, 64), v=z(4, 2, 64))
    with pytest.raises(ValueError):                                         # inv_freq without positions
        rra.qk_norm_rope(z(4, 2, 64), z(4, 2, 64), None, cu, 1, z(4, 2, 64), z(4, 2, 64), torch.zeros(32))
    with pytest.raises(ValueError):                                         # 3 rows for 2 sequences
        rra.attend_cache(z(3, 2, 64), z(2, 8, 2, 64), z(2, 8, 2, 64), cu, z(3, 2, 64), scale=0.125)
    with pytest.raises(ValueError):                                         # float weights
        rra.linear_epilogue(z(4, 64), z(8, 64, dt=torch.float32), cu, 1, z(4, 8))
    with pytest.raises(ValueError):                                         # fewer entries than B + 1
        rra.linear_epilogue(z(4, 64), z(8, 64), cu, 2, z(4, 8))
    with pytest.raises(ValueError):                                         # c of another shape
        rra.linear_epilogue(z(4, 64), z(8, 64), cu, 1, z(4, 16))
