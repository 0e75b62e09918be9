"""rra_rms_norm over its own inputs, with more rows than run at once (needs a GPU): threads then have several rows, and ask
for the next one while they write to this one.  The bounds are test_gpu_rms_norm's."""
from __future__ import annotations

import pytest
import torch

from test_gpu_rms_norm import BF, E4, F32, FP, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [8, 264, 768, 1032, 4096, 6144, 8192, 12296, 16392])
def test_rms_norm_in_place_many_rows(N):
    T = 9001 if N <= 264 else 2801
    _run(T, T + 3, N, BF, E4, BF, True, seed=N, alias=("sum",))
    _run(T, T, N, BF, E4, BF, True, seed=N + 1, alias=("sum_x",))
    _run(T, T, N, FP, FP, F32, True, seed=N + 2, alias=("sum", "y"))
    _run(T, T + 1, N, BF, BF, None, False, seed=N + 3, alias=("y",))
    _run(T, T, N, BF, BF, BF, False, seed=N + 4, alias=("sum", "y"))
