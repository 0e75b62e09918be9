"""What every programmatic dependent of the block operators keeps to, the headers that it is built of among them (CPU).

Such a kernel starts before the kernels ahead of it have finished and waits for them at its head.  Behind that wait it may not read
by a read-only load: one is for memory that nothing writes as long as the kernel lives, and may move ahead of the wait."""
import os
import re

import pytest

from ragged_attention_token_gb300 import build

READ_ONLY = ("__ldg", "ld.global.nc", "__restrict__")


def _plain(text):
    """Without comments and the attributes of kernels."""
    text = re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)
    return re.sub(r"__(?:launch_bounds|cluster_dims)__\([^()]*(?:\([^()]*\)[^()]*)*\)|__grid_constant__", "", text)


def _code(path):
    return _plain(open(path).read())


def _headers(name, seen):
    for h in re.findall(r'#include "([\w.]+\.cuh)"', _code(os.path.join(build.CSRC, name))):
        if h not in seen:
            seen.add(h)
            _headers(h, seen)
    return seen


def _functions(code):
    """(name, what stands before it, body) of each function, outermost first."""
    at = 0
    while m := re.compile(r"\b(\w+)\s*\([^;{}]*\)\s*(?:const\s*)?\{").search(code, at):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[at], 0)
            at += 1
        yield m[1], re.split(r"[;{}]", code[:m.start()])[-1], code[m.end():at]


def _kernels(code):
    return [(name, body) for name, before, body in _functions(code) if "__global__" in before]


def faults(code, headers):
    """What breaks the rule in a source's code, given its headers' codes."""
    out = [w for w in READ_ONLY if w in code]
    for h in headers:
        for name, _, text in _functions(h):
            if re.search(r"\b" + name + r"\b", code):
                out += [f"{name}: {w}" for w in READ_ONLY if w in text]
    for name, text in _kernels(code):
        if not re.search(r"\b(dependent_launch|start_dependent)\(\)", text):
            out.append(f"{name} does not wait")
    return out


def _block_sources():
    return [f for f in sorted(os.listdir(build.CSRC)) if f.endswith(".cu")
            and "ProgrammaticStreamSerialization" in _code(os.path.join(build.CSRC, f)) and "block.cuh" in _headers(f, set())]


def test_all_of_them_are_looked_at():
    assert _block_sources() == ["attend_cache.cu", "attend_paged.cu", "attend_prompt.cu", "linear_epilogue.cu", "qk_norm_rope.cu",
                                "rms_norm.cu"]
    names = {f: {n for n, _ in _kernels(_code(os.path.join(build.CSRC, f)))} for f in _block_sources()}
    assert names["attend_paged.cu"] == {"paged_few_kernel", "paged_chunk_kernel", "paged_join_kernel"}
    assert names["linear_epilogue.cu"] == {"linear_pair_kernel", "linear_mid_kernel", "linear_few_kernel"}
    assert names["rms_norm.cu"] == {"rms_norm_kernel"}


@pytest.mark.parametrize("f", _block_sources())
def test_reads_behind_the_wait(f):
    headers = [_code(os.path.join(build.CSRC, h)) for h in _headers(f, set())]
    assert faults(_code(os.path.join(build.CSRC, f)), headers) == []


def test_the_check_itself():
    kernel = _plain("__global__ void __launch_bounds__(32) k(const int* p) { start_dependent(); if (p[0]) { f(p); } }  // __ldg")
    helper = "__device__ int f(const int* p) { return p[1]; } __device__ int g(const int* p) { return __ldg(p); }"
    assert faults(kernel, [helper]) == []
    assert faults(kernel.replace("start_dependent();", ""), [helper]) == ["k does not wait"]
    assert faults(kernel.replace("p[0]", "__ldg(p)"), [helper]) == ["__ldg"]
    assert faults(kernel.replace("const int* p", "const int* __restrict__ p"), []) == ["__restrict__"]
    assert faults(kernel.replace("f(p)", "g(p)"), [helper]) == ["g: __ldg"]
