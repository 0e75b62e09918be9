"""The README's example of the block in 8 bits over pages, as it stands there (needs a GPU): a chunk of each prompt, then
other new tokens; the sum, the attention and the last layer of each step against the oracle on what they were given."""
import os
import re

import numpy as np
import pytest
import torch

from block_util import check_rows
from oracle import block as OB
from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


def _example() -> str:
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    found = [b for b in re.findall(r"```python\n(.*?)```", open(path).read(), re.S) if "rra.attend_paged(" in b]
    assert len(found) == 1
    return found[0]


def test_the_example_runs_step_by_step():
    g = torch.Generator().manual_seed(3)
    dtype, C, Hq, Hkv, d, page, B = torch.bfloat16, 320, 8, 2, 128, 32, 3
    W = (Hq + 2 * Hkv) * d
    w = torch.randn((W, C), generator=g) / np.sqrt(C)
    ws = w.abs().amax(1) / 448
    ints = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")
    new = lambda *s, dt=dtype: torch.full(s, float("nan"), device="cuda").to(dt)
    table = np.array([[4, 0, 7], [2, 6, -1], [1, 3, 5]], np.int32)
    env = dict(torch=torch, rra=rra, B=B, Hq=Hq, Hkv=Hkv, d=d, wqkv8=(w / ws[:, None]).to(torch.float8_e4m3fn).cuda(),
               wqkv_scale=ws.cuda(), b=(0.1 * torch.randn(W, generator=g)).cuda(),
               wo=(torch.randn((C, Hq * d), generator=g) / np.sqrt(Hq * d)).to(dtype).cuda(),
               n1=(1 + 0.1 * torch.randn(C, generator=g)).cuda(), table=ints(table),
               inv_freq=(10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda(),
               kp=new(8, page, Hkv, d), vp=new(8, page, Hkv, d))
    env["nq"], env["nk"] = (1 + 0.1 * torch.randn((2, d), generator=g)).cuda()
    code = compile(_example(), "README.md", "exec")
    have = np.zeros(B, int)
    rra.get_device_error(clear=True)
    for n in ([70, 33, 20], [1, 1, 60], [1, 0, 1]):
        T = sum(n)
        keys = [np.arange(have[i], have[i] + n[i]) for i in range(B)]
        have = have + np.asarray(n)
        x, res = torch.randn((T, C), generator=g).to(dtype).cuda(), torch.randn((T, C), generator=g).cuda()
        x0, res0 = x.clone(), res.clone()
        env.update(T=T, x=x, res=res, y8=new(T, C).to(torch.float8_e4m3fn), ys=new(T, dt=torch.float32),
                   qkv=new(T, Hq + 2 * Hkv, d), o=new(T, Hq, d), cu=ints(np.concatenate([[0], np.cumsum(n)])),
                   pos=ints(np.concatenate(keys)), kv_len=ints(have), max_new=max(n), max_kv=int(have.max()),
                   slots=ints(np.concatenate([table[i, k // page] * page + k % page for i, k in enumerate(keys)])))
        exec(code, env)
        torch.cuda.synchronize()
        assert rra.get_device_error() == 0
        s64, _ = OB.rms_norm(x0.double().cpu().numpy(), res0.double().cpu().numpy(), None, 1e-6)
        assert np.all(np.abs(res.double().cpu().numpy() - s64) <= 2.0 ** -24 * np.abs(s64))
        at = 0
        q = env["q"]
        for i in range(B):
            k64, v64 = (torch.from_numpy(OB.cached_rows(env[t].double().cpu().numpy(), table[i], int(have[i]))) for t in ("kp", "vp"))
            assert bool(torch.isfinite(k64).all() and torch.isfinite(v64).all())
            if n[i]:
                check_rows(env["o"][at:at + n[i]].cpu(), q[at:at + n[i]].cpu(), k64, v64, d ** -0.5,
                           have[i] - n[i] + np.arange(n[i]), dtype)
            at += n[i]
        o64 = env["o"].double().cpu().numpy().reshape(T, -1)
        y = OB.linear_epilogue(o64, env["wo"].double().cpu().numpy(), None, "none", None, T)
        S = np.abs(o64) @ np.abs(env["wo"].double().cpu().numpy()).T
        assert np.all(np.abs(x.double().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + (Hq * d + 2) * 2.0 ** -23 * S)
