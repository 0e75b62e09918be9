"""Scales of zero (every kept token weighs the same) and below zero, in the image attention's calls (needs a GPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from gpu_util import check_output, oracle_result
from ragged_attention_token_gb300 import rra
from ragged_attention_token_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, -0.125])
@pytest.mark.parametrize("lens", [[40, 197, 0, 1], [300, 577]])
def test_attend_gather_and_attend_take_any_finite_scale(lens, scale):
    case = W.make_custom(len(lens), max(lens), 2, lens, cls=False)
    ref = oracle_result(case)                                        # (its indices; the attention at this scale below)
    q, k, v = (x.cuda() for x in (case.q, case.k, case.v))
    p64 = [oracle.pack_rows(x.double().numpy(), ref["src"]) for x in (case.q, case.k, case.v)]
    want = oracle.unpack(oracle.attend(*p64, ref["cu"], scale), ref["dst"], case.B, case.N)
    cu = torch.from_numpy(ref["cu"]).cuda()
    src = torch.from_numpy(np.asarray(ref["src"], dtype=np.int32)).cuda()
    out = torch.zeros(q.shape, dtype=torch.float32, device="cuda")
    rra.attend_gather(q, k, v, cu, src, out, scale=scale)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    check_output(out.cpu(), case.keep.numpy(), want)
    flat = [x.view(-1, case.H, case.d)[src[:len(ref["src"])].long()].contiguous() for x in (q, k, v)]
    packed = [torch.zeros((case.B * case.N, case.H, case.d), dtype=x.dtype, device="cuda") for x in flat]
    for dst, x in zip(packed, flat):
        dst[:len(x)] = x
    out.zero_()
    rra.attend(*packed, cu, case.B, case.N, out, scale=scale, src_idx=src, N=case.N)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    check_output(out.cpu(), case.keep.numpy(), want)
