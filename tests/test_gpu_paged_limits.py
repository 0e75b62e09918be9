"""rra_attend_paged at the ends of what its documentation allows (needs a GPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_util import nan_fill
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
