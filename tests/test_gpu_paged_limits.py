"""rra_attend_paged at the ends of what its documentation allows (needs a GPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import check_rows, nan_fill
from ragged_attention_token_gb300 import rra
from test_gpu_attend_paged import Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,max_new", [(10, 100), (10, 10), (70, 4000)])
def test_more_new_tokens_than_rows_are_rows_outside(n, max_new):
    """A sequence within max_new whose rows pass cap is one of rows outside [0, cap]; above max_new it is too long."""
    p = Paged([n - 2], [n + 20], 4, 2, 64, 16, torch.bfloat16, seed=n)
    for bound, code in ((max_new, rra.DEVERR_INDEX_RANGE), (n - 1, rra.DEVERR_SEQ_TOO_LONG)):
        nan_fill(p.o)
        p.at = np.asarray([0, n])
        rra.get_device_error(clear=True)
        p.call(max_new=bound)
        torch.cuda.synchronize()
        assert rra.get_device_error(clear=True) == code
        assert bool(torch.isnan(p.o.float()).all())


def test_more_units_than_a_grid_holds():
    """B sequences of Hkv heads past 2^31: all of them may be asked for, whoever has new tokens."""
    B, H, d, at = 65535, 32769, 64, 40000
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(s, generator=g).to(torch.bfloat16) for s in ((1, H, d), (3, H, d), (3, H, d)))
    pool = torch.zeros((1, 2, 16, H, d), dtype=torch.bfloat16, device="cuda")
    pool[0, 0, :3], pool[0, 1, :3] = k.cuda(), v.cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[at] = 3
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[at + 1:] = 1
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    o = nan_fill(torch.empty((1, H, d), dtype=torch.bfloat16, device="cuda"))
    rra.get_device_error(clear=True)
    rra.attend_paged(q.cuda(), pool[:, 0], pool[:, 1], table, lens, cu, B, 1, 3, o, scale=d ** -0.5)
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    got = o.cpu()
    for h in (0, 1, 2047, 16384, 32767, 32768):
        check_rows(got[:, h:h + 1], q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], d ** -0.5, [2], torch.bfloat16)
    assert bool(torch.isfinite(got.float()).all())
