"""What the block operators' sources have to keep to (CPU)."""
import os
import re

from ragged_attention_token_gb300 import build


def test_no_read_only_loads_in_programmatic_dependents():
    """A kernel that starts before the kernels ahead of it have finished (dependent_launch) may not read by __ldg or
    ld.global.nc: those are for memory that nothing writes during the kernel, and may move ahead of the wait."""
    seen = 0
    for path in build.sources():
        text = re.sub(r"//[^\n]*", "", open(path).read())
        if "dependent_launch()" not in text:
            continue
        seen += 1
        assert "__ldg" not in text and "ld.global.nc" not in text, os.path.basename(path)
        assert "__restrict__" not in text, os.path.basename(path)     # const __restrict__ makes them by itself
    assert seen == 4
