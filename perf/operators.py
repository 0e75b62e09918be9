"""What is measured of the operators of a language-model block on packed rows.

Four operators of the library: the linear layer with bias, activation and
residual (`rra.linear_epilogue`), the per-head norms of queries and keys with
the position rotation and the cache write (`rra.qk_norm_rope`), attention over
packed prompts (`rra.attend_prompt`) and attention of new tokens over a cache
(`rra.attend_cache`).  `run` computes them in their plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with `own` set, through
the library; `exact` computes them in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _lib():
    from ragged_attention_token_gb300 import rra
    return rra


# ------------------------------------------------------------------- cases

def _linear(T, K, N, dtype="bf16", out="bf16", act="none", bias=True, residual=False, pad=0, name=None):
    c = dict(op="linear", T=T, K=K, N=N, dtype=dtype, out=out, act=act, bias=bias, residual=residual, pad=pad)
    return dict(c, name=name) if name else c


def _rope(T, Hq, Hkv, d, dtype="bf16", norm=True, rot=0, interleaved=False, maxpos=4096, stretch=1.0, cache_rows=0,
          name=None):
    c = dict(op="rope", T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, norm=norm, rot=rot or d, interleaved=interleaved,
             maxpos=maxpos, stretch=stretch, cache_rows=cache_rows)
    return dict(c, name=name) if name else c


def _prompt(lens, Hq, Hkv, d, dtype="bf16", causal=True, pad=0, name=None):
    c = dict(op="prompt", lens=",".join(map(str, lens)), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, causal=causal, pad=pad)
    return dict(c, name=name) if name else c


def _cache(lens, cap, nq, Hq, Hkv, d, dtype="bf16", name=None):
    c = dict(op="cache", lens=",".join(map(str, lens)), cap=cap, nq=nq, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype)
    return dict(c, name=name) if name else c


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _ragged(count, lo, hi, step=7919):
    """`count` lengths spread over [lo, hi], in no order."""
    return [lo + (i * step + step // 3) % (hi - lo + 1) for i in range(count)]


def listed():
    return [
        # One decoding step of four sequences: the weights are the work.
        _linear(4, 4096, 4096, residual=True, name="linear_tokens4"),
        # The first half of a small encoder's feed-forward block on four pruned images (about 39 tokens each).
        _linear(156, 384, 1536, "fp16", "fp16", "gelu", pad=632, name="linear_serving_gelu"),
        # The query/key/value projection of 64 unpruned images of 197 tokens.
        _linear(12608, 768, 2304, name="linear_qkv_b64"),
        # A large model's feed-forward projection on a batch of prompts.
        _linear(8192, 4096, 16384, act="silu", bias=False, name="linear_large_silu"),
        # One decoding step of sixteen sequences far into their contexts, keys and values into the cache.
        _rope(16, 32, 8, 128, maxpos=131072, stretch=4.0, cache_rows=16 * 1024, name="rope_tokens16_cache"),
        # A pruned image batch: rotation of part of each head, interleaved pairs, no norm.
        _rope(2569, 12, 12, 64, "fp16", norm=False, rot=32, interleaved=True, maxpos=577, name="rope_images"),
        # A batch of prompts of a large model.
        _rope(16411, 32, 8, 128, maxpos=16384, name="rope_prompts"),
        # A few short texts, one of them a single token.
        _prompt([1, 39, 577, 301], 12, 12, 64, "fp16", pad=106, name="prompt_short"),
        # A mixed batch of prompts with grouped heads.
        _prompt([4096, 1, 2500, 777, 3333, 129, 1900, 2049], 32, 8, 128, name="prompt_mixed"),
        # One long document.
        _prompt([16384], 32, 8, 128, name="prompt_long"),
        # Next tokens of four short chats of a small model.
        _cache([39, 197, 130, 64], 577, 1, 12, 12, 64, "fp16", name="cache_short"),
        # Next tokens of a serving batch with contexts of all lengths.
        _cache(_ragged(32, 1, 16384), 16384, 1, 32, 8, 128, name="cache_batch"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "rope", "prompt", "cache"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "linear":
        K, N = 8 * _log_int(rng, 8, 1024), 8 * _log_int(rng, 8, 2048)
        T = _log_int(rng, 1, 16384)
        T = max(1, min(T, 8192 * 4096 * 16384 // (K * N)))
        return _linear(T, K, N, dtype, rng.choice([dtype, dtype, "fp32"]),
                       rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.5,
                       rng.random() < 0.5, rng.choice([0, 0, rng.randrange(1, 300)]))
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    if op == "rope":
        T = _log_int(rng, 1, 16411)
        T = max(1, min(T, 16411 * 40 * 128 // ((Hq + Hkv) * d)))
        rows = T + rng.randrange(0, 4096) if rng.random() < 0.5 else 0
        return _rope(T, Hq, Hkv, d, dtype, rng.random() < 0.7, 16 * rng.randrange(1, d // 16 + 1), rng.random() < 0.5,
                     _log_int(rng, 1, 1 << 20), rng.choice([1.0, 2.0, 8.0]), rows)
    if op == "prompt":
        lens = [_log_int(rng, 1, 16384) for _ in range(rng.randrange(1, 9))]
        while sum(n * n for n in lens) * Hq * d > 16384 * 16384 * 32 * 128:
            lens[lens.index(max(lens))] = max(1, max(lens) // 2)
        return _prompt(lens, Hq, Hkv, d, dtype, rng.random() < 0.8, rng.choice([0, rng.randrange(1, 200)]))
    B = _log_int(rng, 1, 48)
    cap = _log_int(rng, 16, 32768)
    cap = max(16, min(cap, 32 * 16384 * 8 * 128 // (2 * B * Hkv * d)))
    nq = rng.choice([1, 1, 1, 2, 5])
    return _cache([rng.randrange(0, cap + 1) for _ in range(B)], cap, nq, Hq, Hkv, d, dtype)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g, dtype=torch.float32, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _make(case, seed):
    """The inputs alone (the same for `prepare` and `exact`)."""
    g, dt = _gen(seed), _DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "linear":
        T, K, N, cap = case["T"], case["K"], case["N"], case["T"] + case["pad"]
        s["a"] = _randn((cap, K), g, dt)
        s["w"] = _randn((N, K), g, dt, K ** -0.5)
        s["bias"] = _randn((N,), g, scale=0.5) if case["bias"] else None
        s["residual"] = _randn((cap, N), g, _DT[case["out"]]) if case["residual"] else None
        s["cu"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    elif case["op"] == "rope":
        T, Hq, Hkv, d, rot = case["T"], case["Hq"], case["Hkv"], case["d"], case["rot"]
        qkv = _randn((T, Hq + 2 * Hkv, d), g, dt, 1.7)       # a projection's output: one row per token
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["positions"] = torch.randint(0, case["maxpos"], (T,), generator=g, device="cuda", dtype=torch.int32)
        i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * i / rot) / case["stretch"]).float()
        s["rope_scale"] = 1.0 + 0.1 * math.log(case["stretch"])
        s["q_weight"] = 1.0 + _randn((d,), g, scale=0.2) if case["norm"] else None
        s["k_weight"] = 1.0 + _randn((d,), g, scale=0.2) if case["norm"] else None
        s["cu"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        R = case["cache_rows"]
        if R:
            s["rows"] = torch.randperm(R, generator=g, device="cuda")[:T].to(torch.int32)
            s["kc"], s["vc"] = _randn((R, Hkv, d), g, dt), _randn((R, Hkv, d), g, dt)
    elif case["op"] == "prompt":
        lens, Hq, Hkv, d = _lens(case), case["Hq"], case["Hkv"], case["d"]
        cap = sum(lens) + case["pad"]
        qkv = _randn((cap, Hq + 2 * Hkv, d), g, dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    else:
        lens, Hq, Hkv, d = _lens(case), case["Hq"], case["Hkv"], case["d"]
        B = len(lens)
        s["q"] = _randn((B * case["nq"], Hq, d), g, dt)
        s["k"] = torch.randn((B, case["cap"], Hkv, d), generator=g, device="cuda", dtype=dt)
        s["v"] = torch.randn((B, case["cap"], Hkv, d), generator=g, device="cuda", dtype=dt)
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _make(case, seed)
    if case["op"] == "linear":
        s["c"] = torch.empty((case["T"] + case["pad"], case["N"]), dtype=_DT[case["out"]], device="cuda")
    elif case["op"] == "rope":
        s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        if not case["cache_rows"]:
            s["k_out"] = torch.empty(s["k"].shape, dtype=s["k"].dtype, device="cuda")
    else:
        s["o"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    return s


# --------------------------------------------------------------------- run

def _act(x, act):
    if act == "relu":
        return torch.clamp(x, min=0.0)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _plain_linear(s):
    T = s["case"]["T"]
    x = s["a"][:T].float() @ s["w"].float().t()
    if s["bias"] is not None:
        x = x + s["bias"]
    x = _act(x, s["case"]["act"])
    if s["residual"] is not None:
        x = x + s["residual"][:T].float()
    s["c"][:T] = x.to(s["c"].dtype)
    return s["c"][:T]


def _plain_rotate(x, weight, cos, sin, case):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    rot = case["rot"]
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_rope(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = (torch.cos(angle) * s["rope_scale"]).float(), (torch.sin(angle) * s["rope_scale"]).float()
    s["q_out"].copy_(_plain_rotate(s["q"], s["q_weight"], cos, sin, case))
    k = _plain_rotate(s["k"], s["k_weight"], cos, sin, case).to(s["k"].dtype)
    if case["cache_rows"]:
        rows = s["rows"].long()
        s["kc"][rows] = k
        s["vc"][rows] = s["v"]
        return [s["q_out"], s["kc"], s["vc"]]
    s["k_out"].copy_(k)
    return [s["q_out"], s["k_out"]]


def _plain_attention(q, k, v, scale, visible):
    """q [n, Hq, d], k and v [m, Hkv, d], visible [n, m] or None -> fp32 [n, Hq, d]; rows that see nothing are 0."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    out = torch.empty((n, Hq, d), dtype=torch.float32, device=q.device)
    G = Hq // Hkv
    for h in range(Hkv):
        qh = q[:, h * G:(h + 1) * G].float().transpose(0, 1)                  # [G, n, d]
        x = (qh @ k[:, h].float().t()).mul_(scale)                            # [G, n, m]
        if visible is not None:
            x.masked_fill_(~visible, -math.inf)
        x.sub_(x.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
        w = x.sum(-1, keepdim=True)
        o = (x @ v[:, h].float()) / torch.where(w == 0, torch.ones_like(w), w)
        out[:, h * G:(h + 1) * G] = o.transpose(0, 1)
    return out


def _plain_prompt(s):
    case = s["case"]
    a, scale = 0, case["d"] ** -0.5
    for n in _lens(case):
        sl = slice(a, a + n)
        vis = None
        if case["causal"]:
            i = torch.arange(n, device="cuda")
            vis = i[None, :] <= i[:, None]
        s["o"][sl] = _plain_attention(s["q"][sl], s["k"][sl], s["v"][sl], scale, vis).to(s["o"].dtype)
        a += n
    return s["o"][:a]


def _plain_cache(s):
    case = s["case"]
    nq, scale = case["nq"], case["d"] ** -0.5
    for b, n in enumerate(_lens(case)):
        sl = slice(b * nq, (b + 1) * nq)
        if n == 0:
            s["o"][sl] = 0
            continue
        vis = None
        if nq > 1:
            i, j = torch.arange(nq, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
            vis = j < n - (nq - 1 - i)
        s["o"][sl] = _plain_attention(s["q"][sl], s["k"][b, :n], s["v"][b, :n], scale, vis).to(s["o"].dtype)
    return s["o"]


def _own(s):
    rra, case = _lib(), s["case"]
    if case["op"] == "linear":
        act = {"none": rra.ACT_NONE, "relu": rra.ACT_RELU, "gelu": rra.ACT_GELU, "gelu_tanh": rra.ACT_GELU_TANH,
               "silu": rra.ACT_SILU}[case["act"]]
        rra.linear_epilogue(s["a"], s["w"], s["cu"], 1, s["c"], bias=s["bias"], act=act, residual=s["residual"])
        return s["c"][:case["T"]]
    if case["op"] == "rope":
        kw = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], interleaved=case["interleaved"],
                  rope_scale=s["rope_scale"])
        if case["cache_rows"]:
            rra.qk_norm_rope(s["q"], s["k"], s["positions"], s["cu"], 1, s["q_out"], s["kc"], s["inv_freq"], v=s["v"],
                             v_out=s["vc"], kv_rows=s["rows"], **kw)
            return [s["q_out"], s["kc"], s["vc"]]
        rra.qk_norm_rope(s["q"], s["k"], s["positions"], s["cu"], 1, s["q_out"], s["k_out"], s["inv_freq"], **kw)
        return [s["q_out"], s["k_out"]]
    scale = case["d"] ** -0.5
    if case["op"] == "prompt":
        lens = _lens(case)
        rra.attend_prompt(s["q"], s["k"], s["v"], s["cu"], len(lens), max(lens), s["o"], scale=scale,
                          causal=case["causal"])
        return s["o"][:sum(lens)]
    rra.attend_cache(s["q"], s["k"], s["v"], s["kv_len"], s["o"], scale=scale)
    return s["o"]


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "rope": _plain_rope, "prompt": _plain_prompt,
            "cache": _plain_cache}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work

def work(case):
    es = 2
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        eo = 4 if case["out"] == "fp32" else 2
        b = es * (T * K + N * K) + eo * T * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * K * N}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        heads = Hq + Hkv + (Hkv if case["cache_rows"] else 0)
        T = case["T"]
        return {"bytes": 2 * es * T * heads * d + 4 * T, "flops": T * (Hq + Hkv) * (3 * case["rot"] + 4 * d)}
    lens = _lens(case)
    if case["op"] == "prompt":
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": es * sum(lens) * (2 * Hq + 2 * Hkv) * d, "flops": 4 * d * Hq * pairs}
    nq = case["nq"]
    pairs = sum(max(0, n - (nq - 1 - i)) for n in lens for i in range(nq))
    return {"bytes": es * (2 * sum(lens) * Hkv * d + 2 * len(lens) * nq * Hq * d), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------- exact

def _exact_linear(case, s):
    T, K = case["T"], case["K"]
    w = s["w"].double()
    parts = []
    for a in range(0, T, 2048):
        x = torch.einsum("tk,nk->tn", s["a"][a:min(T, a + 2048)].double(), w)
        if s["bias"] is not None:
            x += s["bias"].double()
        act = case["act"]
        if act == "relu":
            x = torch.where(x > 0, x, torch.zeros_like(x))
        elif act == "gelu":
            x = x * 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        elif act == "gelu_tanh":
            x = x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
        elif act == "silu":
            x = x * torch.sigmoid(x)
        if s["residual"] is not None:
            x = x + s["residual"][a:min(T, a + 2048)].double()
        parts.append(x)
    return torch.cat(parts)


def _exact_rope(case, s):
    rot = case["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    turn = torch.polar(torch.full_like(angle, s["rope_scale"]), angle)[:, None, :]          # [T, 1, rot/2]

    def one(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * weight.double()
        head, tail = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
            y = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(*(h.contiguous() for h in head.split(rot // 2, -1))) * turn
            y = torch.cat([z.real, z.imag], -1)
        return torch.cat([y, tail], -1)

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    if not case["cache_rows"]:
        return [q, k]
    kc, vc = s["kc"].double(), s["vc"].double()
    kc.index_copy_(0, s["rows"].long(), k)
    vc.index_copy_(0, s["rows"].long(), s["v"].double())
    return [q, kc, vc]


def _exact_rows(q, k, v, last):
    """One head, q [n, d], keys 0 .. last[i] visible to row i (last[i] < 0: none)."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for a in range(0, q.shape[0], 4096):
        b = min(q.shape[0], a + 4096)
        m = int(last[b - 1]) + 1
        if m <= 0:
            continue
        x = torch.einsum("id,jd->ij", q[a:b], k[:m]) / math.sqrt(q.shape[1])
        la = last[a:b].to(q.device)
        x = torch.where(torch.arange(m, device=q.device)[None, :] <= la[:, None], x, torch.full_like(x, -math.inf))
        ok = la >= 0
        lse = torch.logsumexp(x[ok], -1, keepdim=True)
        out[a:b][ok] = torch.exp(x[ok] - lse) @ v[:m]
    return out


def _exact_attention(case, s):
    Hq, G = case["Hq"], case["Hq"] // case["Hkv"]
    lens, outs, a = _lens(case), [], 0
    for b, n in enumerate(lens):
        if case["op"] == "prompt":
            q, k, v = s["q"][a:a + n], s["k"][a:a + n], s["v"][a:a + n]
            last = torch.arange(n) if case["causal"] else torch.full((n,), n - 1)
            a += n
        else:
            nq = case["nq"]
            q, k, v = s["q"][b * nq:(b + 1) * nq], s["k"][b, :n], s["v"][b, :n]
            last = n - nq + torch.arange(nq)
        o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            o[:, h] = _exact_rows(q[:, h].double(), k[:, h // G].double(), v[:, h // G].double(), last)
        outs.append(o)
    return torch.cat(outs)


def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None          # over about 20 seconds in 64 bits
    s = _make(case, seed)
    if case["op"] == "linear":
        return _exact_linear(case, s)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    return _exact_attention(case, s)
