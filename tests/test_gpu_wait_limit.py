"""The bounded waits of rra_linear_epilogue and rra_attend_prompt (needs a GPU): with a limit set (rra_set_wait_limit)
that runs out, the call records RRA_DEVERR_WAIT_TIMEOUT and returns, and the next normal call is right."""
import pytest
import torch

from ragged_attention_token_gb300 import rra

pytestmark = pytest.mark.gpu


def _linear(cap, K, N, out):
    g = torch.Generator(device="cuda").manual_seed(cap + K + N)
    a, w = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((cap, K), (N, K)))
    c = torch.empty((cap, N), dtype=out, device="cuda")
    cu = torch.tensor([0, cap], dtype=torch.int32, device="cuda")
    return c, lambda: rra.linear_epilogue(a, w, cu, 1, c)


def _prompt(lens, Hq, Hkv, d, causal, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(sum(lens))
    T = sum(lens)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    cu = torch.tensor(at, dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    return o, lambda: rra.attend_prompt(q, k, v, cu, len(lens), max(lens), o, scale=d ** -0.5, causal=causal)


CALLS = {
    "mid": lambda: _linear(64, 4096, 4096, torch.bfloat16),
    "mid_fp32": lambda: _linear(64, 4096, 4096, torch.float32),
    "mid_one_cta": lambda: _linear(200, 512, 16400, torch.float16),
    "pair": lambda: _linear(3000, 1024, 2304, torch.bfloat16),
    "pair_parts": lambda: _linear(3000, 4096, 2304, torch.float32),
    "prompt_heads": lambda: _prompt([2000] * 4, 16, 4, 128, True),
    "prompt_rows": lambda: _prompt([3000, 17, 900] * 2, 16, 16, 64, False),
    "prompt_split": lambda: _prompt([700, 1], 2, 2, 128, True),
    "prompt_split_64": lambda: _prompt([700], 2, 1, 64, False, torch.float16),
}


def _limited(call, cycles):
    """One call under the limit; the device error it left."""
    rra.get_device_error(clear=True)
    old = rra.set_wait_limit(cycles)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        rra.set_wait_limit(old)
    return rra.get_device_error(clear=True)


@pytest.mark.parametrize("name", list(CALLS))
def test_wait_timeout_is_recorded_and_the_next_call_is_right(name):
    out, call = CALLS[name]()
    out.fill_(float("nan"))
    rra.get_device_error(clear=True)
    call()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    want = out.clone()
    assert bool(torch.isfinite(want.float()).all())
    assert _limited(call, 300) == rra.DEVERR_WAIT_TIMEOUT
    out.fill_(float("nan"))
    call()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    assert torch.equal(out, want)
    # A limit that no wait reaches changes nothing.
    out.fill_(float("nan"))
    assert _limited(call, 10 ** 10) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("name", [n for n in CALLS if not n.startswith("mid")])
def test_what_a_call_that_gave_up_wrote_is_right(name):
    """Limits at which some of the waits run out: an element is right, or as it was."""
    out, call = CALLS[name]()
    call()
    torch.cuda.synchronize()
    want = out.clone()
    seen = set()
    for cycles in [400, 700, 1000, 1500, 2000, 2500, 3000, 4000, 5000, 6000, 8000, 12000, 20000]:
        out.fill_(float("nan"))
        seen.add(_limited(call, cycles))
        assert bool(((out == want) | torch.isnan(out)).all()), cycles
    assert rra.DEVERR_WAIT_TIMEOUT in seen


@pytest.mark.parametrize("name", [n for n in CALLS if n.startswith("mid")])
def test_no_cta_joins_the_sums_of_one_that_gave_up(name):
    """A cluster shares K of a tile: where one of its CTAs gave up, the tile is as it was.  The limits go past the time
    of the whole call, and memory traffic ahead of each call spreads the CTAs' times, so that some clusters end in parts."""
    out, call = CALLS[name]()
    call()
    torch.cuda.synchronize()
    want = out.clone()
    busy = torch.zeros(1 << 26, device="cuda")
    seen = set()
    for cycles in [300, *range(5000, 60000, 250), 10 ** 7]:
        out.fill_(float("nan"))
        busy.add_(1.0)
        seen.add(_limited(call, cycles))
        assert bool(((out == want) | torch.isnan(out)).all()), cycles
    assert seen == {0, rra.DEVERR_WAIT_TIMEOUT}


@pytest.mark.parametrize("n", [131064, 131072, 131073])
@pytest.mark.parametrize("d,causal", [(64, False), (128, True)])
def test_a_long_unit_is_no_long_wait(n, d, causal):
    """The bound is for one wait of a block: a sequence whose units take longer than it (a unit walks over a thousand blocks
    of keys, 2 to 4 million cycles) still passes, whether its last block of values ends in a tail or not (the warp
    for the tails idles until then) and whether its last unit has rows for its second tile or not."""
    out, call = _prompt([n], 1, 1, d, causal)
    out.fill_(float("nan"))
    rra.get_device_error(clear=True)
    call()
    torch.cuda.synchronize()
    assert rra.get_device_error() == 0
    want = out.clone()
    assert bool(torch.isfinite(want.float()).all())
    out.fill_(float("nan"))
    assert _limited(call, 500000) == 0
    assert torch.equal(out, want)
