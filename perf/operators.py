"""Workloads of the FP8 layer operators around the paged MLA decode: RMS norm
with the residual's addition, activation quantisation, the matrix product of
e4m3 operands with a scale for each block of 128, and the same product grouped
by expert.

``run`` computes an operator in elementary fp32 torch operations while ``own``
is false, and calls the library while it is true.  An e4m3 result is returned
as a float8 tensor (its values) beside its fp32 scales.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128  # columns that share one scale
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-10  # smallest block maximum a scale is made from
EPS = 1e-6


def listed():
    return [
        # the latent row (512 + 64 wide) of one new token: a product whose time is latency
        {"name": "gemm-latent-1", "op": "gemm", "tokens": 1, "n": 576, "k": 4096, "out": "bf16"},
        # output projection of a 64-request decode step (128 heads x 128): the weights' bytes count
        {"name": "gemm-decode-64", "op": "gemm", "tokens": 64, "n": 4096, "k": 16384, "out": "bf16"},
        # ragged everywhere: a short last block of k, tiles cut on both sides, fp32 results
        {"name": "gemm-odd-333", "op": "gemm", "tokens": 333, "n": 1000, "k": 2000, "out": "fp32"},
        # a prompt's projection: the tensor cores' rate counts
        {"name": "gemm-prompt-8192", "op": "gemm", "tokens": 8192, "n": 8192, "k": 8192, "out": "bf16"},
        # experts of a decode step: a handful of rows each, every active expert's weights are read
        {"name": "grouped-decode-256", "op": "grouped", "tokens": 256, "experts": 64, "active": 60, "n": 4096, "k": 4096,
         "out": "bf16"},
        # few experts, some without a row, odd sizes
        {"name": "grouped-odd-777", "op": "grouped", "tokens": 777, "experts": 7, "active": 4, "n": 328, "k": 1040,
         "out": "bf16"},
        # experts of a prompt
        {"name": "grouped-prompt-16384", "op": "grouped", "tokens": 16384, "experts": 32, "active": 32, "n": 4096,
         "k": 2048, "out": "bf16"},
        # the norm before a single token's projections
        {"name": "norm-1", "op": "norm", "tokens": 1, "dim": 4096, "stride": 4096, "residual": "bf16", "out": "e4m3"},
        # the latent part of a batch's key rows: a slice of wider rows, no residual, bf16 for the cache write
        {"name": "norm-latent-128", "op": "norm", "tokens": 128, "dim": 512, "stride": 576, "residual": "none",
         "out": "bf16"},
        # a prompt's norm: bytes count
        {"name": "norm-prompt-16384", "op": "norm", "tokens": 16384, "dim": 8192, "stride": 8192, "residual": "bf16",
         "out": "e4m3"},
        # between the experts' two products, decode
        {"name": "act-decode-256", "op": "act", "tokens": 256, "dim": 2048, "act": "silu_mul", "out": "e4m3"},
        # the same for a prompt
        {"name": "act-prompt-32768", "op": "act", "tokens": 32768, "dim": 4096, "act": "silu_mul", "out": "e4m3"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "grouped", "norm", "act"])
    if op == "gemm":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "n": _log_int(rng, 16, 8192), "k": 16 * _log_int(rng, 8, 512),
                "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "grouped":
        experts = _log_int(rng, 2, 64)
        active = rng.randint(1, experts)
        return {"op": op, "tokens": _log_int(rng, active, 16384), "experts": experts, "active": active,
                "n": _log_int(rng, 64, 4096), "k": 16 * _log_int(rng, 8, 128), "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "norm":
        dim = _log_int(rng, 64, 8192)
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "dim": dim, "stride": dim + rng.choice([0, 0, 64, 7]),
                "residual": rng.choice(["none", "bf16"]) if dim > 4096 else rng.choice(["none", "bf16", "fp32"]),
                "out": rng.choice(["bf16", "e4m3"])}
    return {"op": op, "tokens": _log_int(rng, 1, 32768), "dim": _log_int(rng, 64, 4096),
            "act": rng.choice(["none", "silu_mul"]), "out": "e4m3"}


def _blocks(n):
    return -(-n // BLOCK)


def _counts(case, seed):
    """Rows of each expert: ``active`` experts own at least one, unevenly."""
    rng = np.random.default_rng([seed, 17])
    experts, active, tokens = case["experts"], case["active"], case["tokens"]
    counts = np.zeros(experts, dtype=np.int64)
    who = rng.permutation(experts)[:active]
    counts[who] = 1 + rng.multinomial(tokens - active, rng.dirichlet(np.full(active, 4.0)))
    return counts


def _activations(tokens, width, gen):
    """bf16-like values with some wide columns, as hidden states have."""
    x = torch.randn(tokens, width, device="cuda", generator=gen)
    return x * (0.5 + 3.0 * torch.rand(width, device="cuda", generator=gen) ** 8)


def _stored_rows(x):
    """e4m3 rows and [blocks, tokens] scales of fp32 rows (the operand of a product)."""
    t, k = x.shape
    g = _blocks(k)
    v = torch.nn.functional.pad(x, (0, g * BLOCK - k)).view(t, g, BLOCK)
    s = v.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (v / s[:, :, None]).reshape(t, g * BLOCK)[:, :k].to(torch.float8_e4m3fn).contiguous()
    return q, s.t().contiguous()


def _stored_weights(e, n, k, gen):
    """e4m3 weights [e, n, k] with a scale for each 128 x 128 block, expert by expert."""
    gn, gk = _blocks(n), _blocks(k)
    q = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(e, gn, gk, device="cuda")
    for i in range(e):
        w = torch.nn.functional.pad(torch.randn(n, k, device="cuda", generator=gen) / math.sqrt(k),
                                    (0, gk * BLOCK - k, 0, gn * BLOCK - n))
        w = w.view(gn, BLOCK, gk, BLOCK)
        s[i] = w.abs().amax((1, 3)).clamp_min(AMAX_FLOOR) / E4M3_MAX
        w = (w / s[i][:, None, :, None]).reshape(gn * BLOCK, gk * BLOCK)
        q[i] = w[:n, :k].to(torch.float8_e4m3fn)
    return q, s


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, t = case["op"], case["tokens"]
    s = {"case": case}
    if op in ("gemm", "grouped"):
        n, k = case["n"], case["k"]
        s["a"], s["a_scales"] = _stored_rows(_activations(t, k, gen))
        s["w"], s["w_scales"] = _stored_weights(case.get("experts", 1), n, k, gen)
        s["out"] = torch.empty(t, n, dtype=_dtype(case["out"]), device="cuda")
        if op == "gemm":
            s["w"], s["w_scales"] = s["w"][0], s["w_scales"][0]
        else:
            counts = _counts(case, seed)
            s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
            s["most"] = int(counts.max())  # the plain form's padding
        return s
    d = case["dim"]
    if op == "norm":
        s["x"] = _activations(t, case["stride"], gen).to(torch.bfloat16)[:, :d]
        s["weight"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(torch.bfloat16)
        s["residual"] = s["residual_out"] = None
        if case["residual"] != "none":
            s["residual"] = (2 * torch.randn(t, d, device="cuda", generator=gen)).to(_dtype(case["residual"]))
            s["residual_out"] = torch.empty_like(s["residual"])
    else:
        s["x"] = _activations(t, d * (2 if case["act"] == "silu_mul" else 1), gen).to(torch.bfloat16)
    s["y"] = torch.empty(t, d, dtype=_dtype(case["out"]), device="cuda")
    s["y_scales"] = torch.empty(_blocks(d), t, device="cuda") if case["out"] == "e4m3" else None
    return s


# ---- plain forms: fp32 throughout, rounded once at the end


def _quantized(v):
    t, d = v.shape
    g = _blocks(d)
    v = torch.nn.functional.pad(v, (0, g * BLOCK - d)).view(t, g, BLOCK)
    scale = v.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    codes = (v * (1.0 / scale)[:, :, None]).view(t, g * BLOCK)[:, :d]
    return [codes.to(torch.float8_e4m3fn).contiguous(), scale.t().contiguous()]


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    outs = [y.to(torch.bfloat16)] if s["y_scales"] is None else _quantized(y)
    return outs + ([] if s["residual"] is None else [h.to(s["residual"].dtype)])


def _plain_act(s):
    v = s["x"].float()
    if s["case"]["act"] == "silu_mul":
        d = s["case"]["dim"]
        v = v[:, :d] / (1.0 + torch.exp(-v[:, :d])) * v[:, d:]
    return _quantized(v)


def _rows_fp32(s):
    return s["a"].float() * s["a_scales"].t().repeat_interleave(BLOCK, 1)[:, :s["a"].shape[1]]


def _weights_fp32(s):
    n, k = s["w"].shape[-2:]
    return s["w"].float() * s["w_scales"].repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _plain_gemm(s):
    return [(_rows_fp32(s) @ _weights_fp32(s).t()).to(s["out"].dtype)]


def _plain_grouped(s):
    a, off = _rows_fp32(s), s["offsets"].long()
    at = torch.arange(a.shape[0], device="cuda")
    padded = (off[:-1, None] + torch.arange(s["most"], device="cuda")).clamp_max(a.shape[0] - 1)
    out = torch.bmm(a[padded], _weights_fp32(s).transpose(1, 2))
    expert = torch.searchsorted(off[1:], at, right=True)
    return [out[expert, at - off[expert]].to(s["out"].dtype)]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "act": _plain_act, "gemm": _plain_gemm, "grouped": _plain_grouped}[op](s)
    from paged_mla_decode_08_gb300 import binding as B

    if op == "gemm":
        out_dtype = B.MLA_OUT_FP32 if s["case"]["out"] == "fp32" else B.MLA_OUT_BF16
        B.mla_gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], out_dtype)
        return [s["out"]]
    if op == "grouped":
        out_dtype = B.MLA_OUT_FP32 if s["case"]["out"] == "fp32" else B.MLA_OUT_BF16
        B.mla_grouped_gemm_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["offsets"], s["out"], out_dtype)
        return [s["out"]]
    y_dtype = B.MLA_OUT_BF16 if s["case"]["out"] == "bf16" else B.MLA_OUT_E4M3
    outs = [s["y"]] if s["y_scales"] is None else [s["y"], s["y_scales"]]
    if op == "norm":
        res_dtype = B.MLA_OUT_FP32 if s["case"]["residual"] == "fp32" else B.MLA_OUT_BF16
        B.mla_add_rmsnorm(s["x"], s["residual"], s["residual_out"], res_dtype, s["weight"], EPS, s["y"], y_dtype,
                          s["y_scales"])
        return outs + ([] if s["residual"] is None else [s["residual_out"]])
    act = B.MLA_ACT_SILU_MUL if s["case"]["act"] == "silu_mul" else B.MLA_ACT_NONE
    B.mla_act_quantize(s["x"], act, s["y"], y_dtype, s["y_scales"])
    return outs


def work(case):
    op, t = case["op"], case["tokens"]
    if op in ("gemm", "grouped"):
        n, k, g = case["n"], case["k"], _blocks(case["k"])
        weights = case.get("active", 1) * (n * k + 4 * _blocks(n) * g)
        index = 4 * (case["experts"] + 1) if op == "grouped" else 0
        return {"bytes": t * k + 4 * t * g + weights + index + t * n * (4 if case["out"] == "fp32" else 2),
                "flops": 2 * t * n * k}
    d = case["dim"]
    out = t * d * 2 if case["out"] == "bf16" else t * d + 4 * t * _blocks(d)
    if op == "norm":
        residual = {"none": 0, "bf16": 2, "fp32": 4}[case["residual"]]
        return {"bytes": t * d * (2 + 2 * residual) + 2 * d + out, "flops": 6 * t * d}
    wide = 2 if case["act"] == "silu_mul" else 1
    return {"bytes": 2 * t * d * wide + out, "flops": (8 if wide == 2 else 3) * t * d}


# ---- the definitions in 64 bits


def _e4m3_nearest(v):
    """Nearest e4m3 value of fp64 values within +-448, ties to even."""
    exponent = torch.frexp(v.abs().clamp_min(2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def _exact_quantized(v):
    codes, scales = [], []
    for c in range(0, v.shape[1], BLOCK):
        part = v[:, c:c + BLOCK]
        scale = torch.clamp(part.abs().max(dim=1).values, min=AMAX_FLOOR) / E4M3_MAX
        codes.append(_e4m3_nearest(part / scale[:, None]))
        scales.append(scale)
    return [torch.cat(codes, 1), torch.stack(scales)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h += s["residual"].double()
        rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["dim"] + EPS)
        y = s["weight"].double() * (h / rms)
        outs = [y] if case["out"] == "bf16" else _exact_quantized(y)
        return outs + ([] if s["residual"] is None else [h])
    if op == "act":
        v = s["x"].double()
        if case["act"] == "silu_mul":
            gate, up = v.chunk(2, dim=1)
            v = gate * torch.sigmoid(gate) * up
        return _exact_quantized(v)
    t, n, k = case["tokens"], case["n"], case["k"]
    rows = [0, t] if op == "gemm" else s["offsets"].tolist()
    w, sw = (s["w"][None], s["w_scales"][None]) if op == "gemm" else (s["w"], s["w_scales"])
    out = torch.zeros(t, n, dtype=torch.float64, device="cuda")
    of_row = torch.arange(n, device="cuda") // BLOCK
    for e, (lo, hi) in enumerate(zip(rows[:-1], rows[1:])):
        if hi > lo:
            for b in range(_blocks(k)):
                cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
                part = s["a"][lo:hi, cols].double() @ w[e, :, cols].double().t()
                out[lo:hi] += part * s["a_scales"][b, lo:hi, None].double() * sw[e, :, b][of_row].double()
    return [out]
