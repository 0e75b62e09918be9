"""The README's example of a language model's block, as it stands there (needs a GPU): prompts, then one more token of
each sequence against the cache that the prompts filled, both against the oracle."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


def _example() -> str:
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    blocks = re.findall(r"```python\n(.*?)```", open(path).read(), re.S)
    found = [b for b in blocks if "rra.attend_cache(" in b]
    assert len(found) == 1
    return found[0]


def test_the_decoding_step_finds_the_prompts_in_the_cache():
    g = torch.Generator().manual_seed(3)
    dtype, C, Hq, Hkv, d, lens, cap = torch.bfloat16, 320, 8, 2, 128, [70, 1, 33], 96
    B, T, W = len(lens), sum(lens), (Hq + 2 * Hkv) * d
    full = [n + 1 for n in lens]
    at = np.concatenate([[0], np.cumsum(full)])
    prompt_rows = np.concatenate([np.arange(at[i], at[i] + n) for i, n in enumerate(lens)])
    x_full = torch.randn((sum(full), C), generator=g).to(dtype)
    wqkv = (torch.randn((W, C), generator=g) / np.sqrt(C)).to(dtype)
    wo = (torch.randn((C, Hq * d), generator=g) / np.sqrt(Hq * d)).to(dtype)
    b = 0.1 * torch.randn(W, generator=g)
    nq, nk = 1 + 0.1 * torch.randn((2, d), generator=g)
    inv_freq = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float()

    def ints(v):
        return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")

    def new(*shape):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

    env = dict(
        torch=torch, rra=rra, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, cap=cap, max_seqlen=max(lens),
        x=x_full[prompt_rows].cuda(), x1=x_full[at[1:] - 1].cuda(), wqkv=wqkv.cuda(), wo=wo.cuda(), b=b.cuda(),
        nq=nq.cuda(), nk=nk.cuda(), inv_freq=inv_freq.cuda(), qkv=new(T, Hq + 2 * Hkv, d), qkv1=new(B, Hq + 2 * Hkv, d),
        o=new(T, Hq, d), o1=new(B, Hq, d), kc=torch.zeros((B * cap, Hkv, d), dtype=dtype, device="cuda"),
        vc=torch.zeros((B * cap, Hkv, d), dtype=dtype, device="cuda"), cu=ints(np.concatenate([[0], np.cumsum(lens)])),
        cu1=ints(np.arange(B + 1)), pos=ints(np.concatenate([np.arange(n) for n in lens])), pos1=ints(lens),
        slots=ints(np.concatenate([i * cap + np.arange(n) for i, n in enumerate(lens)])),
        slots1=ints([i * cap + n for i, n in enumerate(lens)]), kv_len=ints(full))
    rra.get_device_error(clear=True)
    exec(compile(_example(), "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0

    x64 = x_full.double().numpy()
    qkv = OB.linear_epilogue(x64, wqkv.double().numpy(), b.double().numpy(), "none", None, len(x64)).reshape(-1, Hq + 2 * Hkv, d)
    p64 = np.concatenate([np.arange(n) for n in full])
    q = OB.norm_rope(qkv[:, :Hq], p64, nq.double().numpy(), 1e-6, inv_freq.double().numpy(), False, 1.0)
    k = OB.norm_rope(qkv[:, Hq:Hq + Hkv], p64, nk.double().numpy(), 1e-6, inv_freq.double().numpy(), False, 1.0)
    o = np.concatenate([OB.attend_rows(q[at[i]:at[i + 1]], k[at[i]:at[i + 1]], qkv[at[i]:at[i + 1], Hq + Hkv:], d ** -0.5,
                                       np.arange(full[i]))[0] for i in range(B)])
    y = OB.linear_epilogue(o.reshape(-1, Hq * d), wo.double().numpy(), None, "none", x64, len(x64))
    # Four roundings on the way, each at most half a step of values of order one to five, through sums whose weights'
    # squares add up to one, and the last rounding: within 24 half steps of 1 + |y|.
    u = torch.finfo(dtype).eps / 2
    for name, rows in (("x", prompt_rows), ("x1", at[1:] - 1)):
        err = np.abs(env[name].cpu().double().numpy() - y[rows])
        assert np.all(err <= 24 * u * (1 + np.abs(y[rows]))), (name, float(err.max()))
