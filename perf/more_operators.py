"""Workloads of the operators that a prompt needs over the latent cache: the
table of scaled rotary positions, the rotation, the gather of cached rows, latent
attention in its expanded form, and the merge of two partial results.

``run`` computes an operator in elementary torch operations while ``own`` is
false, and calls the library while it is true.
"""

import math

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
BLOCK = 128  # latent columns that share one scale
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-10
BASE = 10000.0
BETA_FAST, BETA_SLOW = 32.0, 1.0


def listed():
    return [
        # a short prompt on one of eight shards of the heads: latency
        {"name": "attn-short-130", "op": "attn", "heads": 16, "q_lens": "130", "k_lens": "130", "causal": True},
        # prompts that arrive together, one with a cached prefix, one without a new token, one of a single token
        {"name": "attn-ragged-8", "op": "attn", "heads": 128, "q_lens": "1537,1,700,0,260,1100,64,333",
         "k_lens": "1537,1,2800,77,260,1100,64,333", "causal": True},
        # a chunk of new tokens over its cached prefix: every key is visible, few rows, long keys
        {"name": "attn-prefix-20000", "op": "attn", "heads": 16, "q_lens": "500", "k_lens": "20000", "causal": False},
        # one long prompt, all heads: the tensor cores' rate counts
        {"name": "attn-prompt-8192", "op": "attn", "heads": 128, "q_lens": "8192", "k_lens": "8192", "causal": True},
        # the rotary parts of a handful of new tokens
        {"name": "rope-8", "op": "rope", "tokens": 8, "heads": 16, "rotary": 64, "neox": False, "positions": 4096},
        # ... and of a prompt, slices of 192-wide heads and of 576-wide rows: bytes count
        {"name": "rope-prompt-8192", "op": "rope", "tokens": 8192, "heads": 128, "rotary": 64, "neox": False,
         "positions": 131072},
        # the table of a short context, unscaled
        {"name": "table-4096", "op": "table", "positions": 4096, "first": 0, "rotary": 64, "scaling": "none",
         "factor": 1.0, "original": 4096, "magnitude": 1.0},
        # the table of a long context, stretched forty times
        {"name": "table-yarn-163840", "op": "table", "positions": 163840, "first": 0, "rotary": 64, "scaling": "yarn",
         "factor": 40.0, "original": 4096, "magnitude": 1.0},
        # a short prefix of a bf16 cache, for a bf16 expansion
        {"name": "gather-bf16-300", "op": "gather", "lens": "130,1,0,169", "starts": "0,64,5,31", "page": 32,
         "cache": "bf16", "latent": "bf16"},
        # a chunk of a long prefix of an FP8 cache, for an FP8 expansion
        {"name": "gather-e4m3-65536", "op": "gather", "lens": "30000,20001,7,15528", "starts": "0,64,1000,12345", "page": 64,
         "cache": "e4m3", "latent": "e4m3"},
        # the two partial results of a few rows
        {"name": "merge-8", "op": "merge", "tokens": 8, "heads": 16, "dim": 128},
        # ... and of a long prompt's chunk
        {"name": "merge-8192", "op": "merge", "tokens": 8192, "heads": 128, "dim": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ints(text):
    return [int(v) for v in text.split(",")]


def _text(values):
    return ",".join(str(v) for v in values)


MOST_PAIRS = 8192 * 8193 // 2 * 128  # visible (row, key, head) triples of the largest listed case


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "table", "gather", "merge"])
    if op == "attn":
        batch, causal = _log_int(rng, 1, 16), rng.random() < 0.6
        tokens = _log_int(rng, 1, 8192)
        share = [rng.expovariate(1.0) for _ in range(batch)]
        q = [int(tokens * s / sum(share)) for s in share]
        q[rng.randrange(batch)] += tokens - sum(q)
        if causal:  # new tokens, some behind a prefix
            k = [n + (_log_int(rng, 1, 4096) if rng.random() < 0.4 else 0) for n in q]
        else:
            k = [_log_int(rng, 1, 16384 // batch + 1) if rng.random() < 0.9 else 0 for _ in q]
        pairs = sum(_visible(n, m, causal) for n, m in zip(q, k))
        whole = sum(n * m for n, m in zip(q, k))  # what the plain form computes
        heads = min(_log_int(rng, 1, 128), max(1, MOST_PAIRS // max(1, pairs)), max(1, 2 * MOST_PAIRS // max(1, whole)))
        return {"op": op, "heads": heads, "q_lens": _text(q), "k_lens": _text(k), "causal": causal}
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "heads": _log_int(rng, 1, 128),
                "rotary": rng.choice([64, 64, 32, 40]), "neox": rng.random() < 0.5, "positions": _log_int(rng, 16, 131072)}
    if op == "table":
        scaling = rng.choice(["none", "linear", "yarn"])
        return {"op": op, "positions": _log_int(rng, 512, 131072), "first": rng.choice([0, 0, 1000, 500001]),
                "rotary": rng.choice([64, 64, 32, 40]), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else round(rng.uniform(1.5, 40.0), 2),
                "original": rng.choice([2048, 4096, 8192]), "magnitude": 1.0 if scaling != "yarn" else
                round(rng.uniform(0.8, 1.4), 3)}
    if op == "gather":
        batch = _log_int(rng, 1, 32)
        tokens = _log_int(rng, 1, 65536)
        share = [rng.expovariate(1.0) for _ in range(batch)]
        lens = [int(tokens * s / sum(share)) for s in share]
        lens[rng.randrange(batch)] += tokens - sum(lens)
        return {"op": op, "lens": _text(lens), "starts": _text([rng.randint(0, 2000) for _ in lens]),
                "page": rng.choice([32, 64]), "cache": rng.choice(["bf16", "e4m3"]), "latent": rng.choice(["bf16", "e4m3"])}
    dim = rng.choice([128, 128, 512, 72])
    return {"op": op, "tokens": _log_int(rng, 1, 8192), "heads": _log_int(rng, 1, 128 * 128 // max(dim, 128)), "dim": dim}


def _visible(n, m, causal):
    """Visible pairs of n queries at the end of m keys."""
    if not causal:
        return n * m
    rows = min(n, m)  # queries that see a key
    return rows * (m - rows + m + 1) // 2


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _frequencies(case):
    """Turns of 2 pi per position, in 64 bits."""
    r = case["rotary"]
    f = [BASE ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        f = [w / case["factor"] for w in f]
    if case["scaling"] == "yarn":
        at = lambda beta: r * math.log(case["original"] / (beta * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(at(BETA_FAST)), 0), min(math.ceil(at(BETA_SLOW)), r - 1)
        hi = hi + 0.001 if hi == lo else hi
        g = [min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(r // 2)]
        f = [w / case["factor"] * b + w * (1.0 - b) for w, b in zip(f, g)]
    return f


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=gen)  # noqa: E731
    s, op = {"case": case}, case["op"]
    bf16 = torch.bfloat16
    if op == "attn":
        h, q_lens, k_lens = case["heads"], _ints(case["q_lens"]), _ints(case["k_lens"])
        cu_q, cu_k = _cu(q_lens), _cu(k_lens)
        tq, tk = cu_q[-1], cu_k[-1]
        gain = 0.5 + 2.0 * rand(h, 1)  # heads that look around and heads that look at few keys
        q = (randn(tq, h, NOPE + ROPE) * gain).to(bf16)
        kv = randn(tk, h, NOPE + VDIM)
        firsts = torch.tensor([a for a, n in zip(cu_k, k_lens) if n], dtype=torch.long, device="cuda")
        kv[firsts, :, :NOPE] *= 3.0  # a request's first key draws attention
        kv = kv.to(bf16)
        s.update(q_nope=q[..., :NOPE], q_pe=q[..., NOPE:], k_nope=kv[..., :NOPE], v=kv[..., NOPE:],
                 k_pe=randn(tk, ROPE).to(bf16), q_lens=q_lens, k_lens=k_lens,
                 cu_q=torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                 cu_k=torch.tensor(cu_k, dtype=torch.int32, device="cuda"),
                 out=torch.empty(tq, h, VDIM, dtype=bf16, device="cuda"), lse=torch.empty(tq, h, device="cuda"))
        s["workspace"] = None
        if own:
            from paged_mla_decode_08_gb300 import binding as B

            need = B.mla_prefill_workspace_bytes(tq, tk, len(q_lens), h)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    elif op == "rope":
        t, h, r = case["tokens"], case["heads"], case["rotary"]
        s["q"] = randn(t, h, NOPE + r).to(bf16)[..., NOPE:]
        s["k"] = randn(t, LATENT + r).to(bf16)[:, LATENT:]
        first = int(torch.randint(0, max(1, case["positions"] - t + 1), (1,), device="cuda", generator=gen))
        s["pos"] = (first + torch.arange(t, device="cuda")) % case["positions"]
        ang = torch.arange(case["positions"], device="cuda").double()[:, None] * torch.tensor(
            [BASE ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["q_out"] = torch.empty(t, h, r, dtype=bf16, device="cuda")
        s["k_out"] = torch.empty(t, r, dtype=bf16, device="cuda")
    elif op == "table":
        # no tensor goes in: another seed is another window of positions
        s["first"] = case["first"] + int(torch.randint(0, 1000, (1,), device="cuda", generator=gen))
        s["table"] = torch.empty(case["positions"], case["rotary"], device="cuda")
    elif op == "gather":
        lens, starts, page = _ints(case["lens"]), _ints(case["starts"]), case["page"]
        blocks = [-(-(a + n) // page) for a, n in zip(starts, lens)]
        pool, width = sum(blocks) + 3, max(blocks) + 1
        order = torch.randperm(pool, device="cuda", generator=gen).to(torch.int32)
        s["block_table"] = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
        for b, (n, at) in enumerate(zip(blocks, _cu(blocks))):
            s["block_table"][b, :n] = order[at:at + n]
        rows = randn(pool, page, LATENT + ROPE)
        rows[..., LATENT:] *= 4.0
        s["kv"] = (rows * 8.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) if case["cache"] == "e4m3" else rows.to(bf16)
        s["k_scale"] = 0.125 * 1.1 if case["cache"] == "e4m3" else 1.0
        s["lens"], t = lens, sum(lens)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
        s["latent"] = torch.empty(t, LATENT, dtype=torch.float8_e4m3fn if case["latent"] == "e4m3" else bf16, device="cuda")
        s["scales"] = torch.empty(LATENT // BLOCK, t, device="cuda") if case["latent"] == "e4m3" else None
        s["k_pe"] = torch.empty(t, ROPE, dtype=bf16, device="cuda")
    else:
        t, h, d = case["tokens"], case["heads"], case["dim"]
        for x in "ab":
            s["out_" + x] = randn(t, h, d).to(bf16)
            s["lse_" + x] = 6.0 + 2.0 * randn(t, h)
        s["lse_b"][rand(t, h) < 0.05] = -math.inf  # rows without a key in the second part
        s["out_b"][torch.isinf(s["lse_b"])] = 0
        s["out"], s["lse"] = torch.empty_like(s["out_a"]), torch.empty_like(s["lse_a"])
    return s


# ---- plain forms: fp32 throughout (angles in 64 bits), rounded once at the end


def _plain_attn(s):
    tq, h = s["q_nope"].shape[:2]
    out = torch.zeros(tq, h, VDIM, device="cuda")
    lse = torch.full((tq, h), -math.inf, device="cuda")
    cq = ck = 0
    for n, m in zip(s["q_lens"], s["k_lens"]):
        step = max(1, (1 << 29) // max(1, n * m))  # heads at a time
        if n and m:
            dead = None
            if s["case"]["causal"]:
                dead = torch.arange(m, device="cuda")[None, :] > torch.arange(n, device="cuda")[:, None] + (m - n)
            for lo in range(0, h, step):
                hs = slice(lo, lo + step)
                q = torch.cat([s["q_nope"][cq:cq + n, hs], s["q_pe"][cq:cq + n, hs]], 2).float().transpose(0, 1)
                k_pe = s["k_pe"][ck:ck + m, None].expand(m, q.shape[0], ROPE)
                k = torch.cat([s["k_nope"][ck:ck + m, hs], k_pe], 2).float().transpose(0, 1)
                x = (q @ k.transpose(1, 2)).mul_(SCALE)
                if dead is not None:
                    x.masked_fill_(dead, -math.inf)
                top = x.amax(2, keepdim=True).clamp_min(-3e38)
                x.sub_(top).exp_()
                total = x.sum(2, keepdim=True)
                part = (x @ s["v"][ck:ck + m, hs].float().transpose(0, 1)) / total.clamp_min(1e-38)
                out[cq:cq + n, hs] = part.transpose(0, 1)
                lse[cq:cq + n, hs] = (top + total.log())[..., 0].t()
        cq, ck = cq + n, ck + m
    return [out.to(torch.bfloat16), lse]


def _plain_rope(s):
    r = s["case"]["rotary"]
    cs = s["table"][s["pos"]]
    outs = []
    for x, c, sn in ((s["q"], cs[:, None, :r // 2], cs[:, None, r // 2:]), (s["k"], cs[:, :r // 2], cs[:, r // 2:])):
        x = x.float()
        if s["case"]["neox"]:
            a, b = x[..., :r // 2], x[..., r // 2:]
            y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        outs.append(y.to(torch.bfloat16))
    return outs


def _plain_table(s):
    case = s["case"]
    pos = torch.arange(s["first"], s["first"] + case["positions"], device="cuda", dtype=torch.float64)
    ang = pos[:, None] * torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    return [(torch.cat([ang.cos(), ang.sin()], 1) * case["magnitude"]).float()]


def _plain_gather(s):
    page, width = s["kv"].shape[1:]
    tokens = int(s["latent"].shape[0])
    at = torch.arange(tokens, device="cuda")
    req = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    tok = s["starts"].long()[req] + at - s["cu"].long()[req]
    slot = s["block_table"].long()[req, tok // page] * page + tok % page
    rows = s["kv"].view(-1, width)[slot]
    k_pe = (rows[:, LATENT:].float() * s["k_scale"]).to(torch.bfloat16)
    if s["scales"] is None:
        return [(rows[:, :LATENT].float() * s["k_scale"]).to(torch.bfloat16), k_pe]
    if s["case"]["cache"] == "e4m3":  # the stored codes with the cache's scale
        return [rows[:, :LATENT].contiguous(), torch.full((LATENT // BLOCK, tokens), s["k_scale"], device="cuda"), k_pe]
    v = rows[:, :LATENT].float().view(tokens, -1, BLOCK)
    scale = v.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    codes = (v * (1.0 / scale)[:, :, None]).view(tokens, LATENT).to(torch.float8_e4m3fn)
    return [codes, scale.t().contiguous(), k_pe]


def _plain_merge(s):
    a, b = s["lse_a"], s["lse_b"]
    top = torch.maximum(a, b).clamp_min(-3e38)
    wa, wb = torch.exp(a - top), torch.exp(b - top)
    total = wa + wb
    wa, wb = wa / total.clamp_min(1e-38), wb / total.clamp_min(1e-38)
    out = s["out_a"].float() * wa[..., None] + s["out_b"].float() * wb[..., None]
    return [out.to(torch.bfloat16), top + total.log()]


def run(state):
    s, case, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "rope": _plain_rope, "table": _plain_table, "gather": _plain_gather,
                "merge": _plain_merge}[op](s)
    from paged_mla_decode_08_gb300 import binding as B

    if op == "attn":
        B.mla_prefill(s["q_nope"], s["q_pe"], s["k_nope"], s["k_pe"], s["v"], s["cu_q"], s["cu_k"], case["causal"], SCALE,
                      s["out"], s["lse"], s["workspace"])
        return [s["out"], s["lse"]]
    if op == "rope":
        B.mla_rope(s["q"], s["k"], s["pos"], s["table"], case["neox"], s["q_out"], s["k_out"])
        return [s["q_out"], s["k_out"]]
    if op == "table":
        scaling = {"none": B.MLA_ROPE_PLAIN, "linear": B.MLA_ROPE_LINEAR, "yarn": B.MLA_ROPE_YARN}[case["scaling"]]
        B.mla_rope_table(s["table"], s["first"], BASE, scaling, case["factor"], case["original"], BETA_FAST, BETA_SLOW,
                         case["magnitude"])
        return [s["table"]]
    if op == "gather":
        cache = B.MLA_KV_E4M3 if case["cache"] == "e4m3" else B.MLA_KV_BF16
        latent = B.MLA_OUT_E4M3 if case["latent"] == "e4m3" else B.MLA_OUT_BF16
        B.mla_cache_gather(s["kv"], cache, s["block_table"], s["starts"], s["cu"], s["k_scale"], s["latent"], latent,
                           s["scales"], s["k_pe"])
        return [s["latent"]] + ([] if s["scales"] is None else [s["scales"]]) + [s["k_pe"]]
    B.mla_merge_states(s["out_a"], s["lse_a"], s["out_b"], s["lse_b"], s["out"], s["lse"])
    return [s["out"], s["lse"]]


def work(case):
    op = case["op"]
    if op == "attn":
        h, q, k = case["heads"], _ints(case["q_lens"]), _ints(case["k_lens"])
        tq, tk = sum(q), sum(m for n, m in zip(q, k) if n)  # keys without a query are not needed
        pairs = sum(_visible(n, m, case["causal"]) for n, m in zip(q, k))
        return {"bytes": tq * h * (2 * (NOPE + ROPE + VDIM) + 4) + tk * (2 * h * (NOPE + VDIM) + 2 * ROPE) + 8 * (len(q) + 1),
                "flops": 2 * (NOPE + ROPE + VDIM) * h * pairs}
    if op == "rope":
        t, r, rows = case["tokens"], case["rotary"], case["heads"] + 1
        return {"bytes": t * (4 * r * rows + 8) + 4 * r * min(t, case["positions"]), "flops": 3 * t * r * rows}
    if op == "table":
        n = case["positions"] * case["rotary"]
        return {"bytes": 4 * n, "flops": 20 * n}
    if op == "gather":
        t = sum(_ints(case["lens"]))
        read = (LATENT + ROPE) * (1 if case["cache"] == "e4m3" else 2)
        write = (LATENT + 4 * LATENT // BLOCK if case["latent"] == "e4m3" else 2 * LATENT) + 2 * ROPE
        return {"bytes": t * (read + write) + 4 * sum(-(-n // case["page"]) for n in _ints(case["lens"])),
                "flops": t * (LATENT + ROPE)}
    rows = case["tokens"] * case["heads"]
    return {"bytes": rows * (6 * case["dim"] + 12), "flops": rows * (3 * case["dim"] + 10)}


# ---- the definitions in 64 bits


def _exact_attn(case, s):
    h = case["heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        keys = slice(cu_k[b], cu_k[b + 1])
        for head in range(h if m else 0):
            kn, kp, v = s["k_nope"][keys, head].double(), s["k_pe"][keys].double(), s["v"][keys, head].double()
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)
                rows = slice(cu_q[b] + lo, cu_q[b] + hi)
                seen = max(0, m - n + hi) if case["causal"] else m  # keys that some of these rows see
                if not seen:
                    continue
                x = SCALE * (s["q_nope"][rows, head].double() @ kn[:seen].T + s["q_pe"][rows, head].double() @ kp[:seen].T)
                if case["causal"]:
                    last = m - n + torch.arange(lo, hi, device="cuda")
                    x[torch.arange(seen, device="cuda")[None] > last[:, None]] = -math.inf
                z = torch.logsumexp(x, 1)
                weights = torch.exp(x - z[:, None]).nan_to_num_(0.0)
                out[rows, head], lse[rows, head] = weights @ v[:seen], z
    return [out, lse]


def _exact_codes(v):
    """Nearest e4m3 values (ties to even) and scales of fp64 rows."""
    codes, scales = torch.empty_like(v), []
    for c in range(0, v.shape[1], BLOCK):
        part = v[:, c:c + BLOCK]
        scale = part.abs().max(1).values.clamp(min=AMAX_FLOOR) / E4M3_MAX
        w = part / scale[:, None]
        step = torch.ldexp(torch.ones_like(w), torch.frexp(w.abs().clamp_min(2.0 ** -6))[1] - 4)
        codes[:, c:c + BLOCK] = torch.round(w / step) * step
        scales.append(scale)
    return codes, torch.stack(scales)


def _exact_gather(case, s):
    page, table = case["page"], s["block_table"].tolist()
    slots = [table[b][tok // page] * page + tok % page
             for b, (a, n) in enumerate(zip(_ints(case["starts"]), _ints(case["lens"]))) for tok in range(a, a + n)]
    rows = s["kv"].view(-1, LATENT + ROPE)[torch.tensor(slots, dtype=torch.long, device="cuda")].double()
    k_pe = rows[:, LATENT:] * s["k_scale"]
    if case["latent"] == "bf16":
        return [rows[:, :LATENT] * s["k_scale"], k_pe]
    if case["cache"] == "bf16":
        return [*_exact_codes(rows[:, :LATENT]), k_pe]
    scale = torch.full((LATENT // BLOCK, len(slots)), s["k_scale"], dtype=torch.float64, device="cuda")
    return [rows[:, :LATENT], scale, k_pe]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "attn":
        return _exact_attn(case, s)
    if op == "gather":
        return _exact_gather(case, s)
    if op == "table":
        p = s["first"] + torch.arange(case["positions"], device="cuda").double()
        w = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        turn = torch.outer(p, w)
        return [case["magnitude"] * torch.cat([torch.cos(turn), torch.sin(turn)], 1)]
    if op == "rope":
        half = case["rotary"] // 2
        cs = s["table"].double().index_select(0, s["pos"])
        turn = torch.complex(cs[:, :half], cs[:, half:])
        outs = []
        for x, w in ((s["q"].double(), turn[:, None]), (s["k"].double(), turn)):
            pairs = x.unflatten(-1, (2, half)).transpose(-1, -2) if case["neox"] else x.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
            outs.append((z.transpose(-1, -2) if case["neox"] else z).flatten(-2))
        return outs
    z = torch.logaddexp(s["lse_a"].double(), s["lse_b"].double())
    parts = [torch.exp(s["lse_" + x].double() - z)[..., None] * s["out_" + x].double() for x in "ab"]
    return [parts[0] + parts[1], z]
