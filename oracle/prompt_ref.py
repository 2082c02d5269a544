"""Float64 oracle of the prompt's operators: rotary table, rotation, cache gather,
expanded attention, merge.  Inputs are the stored values as float64 arrays."""

import numpy as np


def rope_frequencies(dim, base, scaling="plain", factor=1.0, original=4096, beta_fast=32.0, beta_slow=1.0):
    """Angle of one position for each pair."""
    f = base ** (-2.0 * np.arange(dim // 2) / dim)
    if scaling == "linear":
        return f / factor
    if scaling == "yarn":
        def pair(beta):
            return dim * np.log(original / (2 * np.pi * beta)) / (2 * np.log(base))

        lo, hi = max(np.floor(pair(beta_fast)), 0.0), min(np.ceil(pair(beta_slow)), dim - 1.0)
        g = np.clip((np.arange(dim // 2) - lo) / (hi - lo if hi != lo else 0.001), 0.0, 1.0)
        return f / factor * g + f * (1 - g)
    return f


def rope_table(first, positions, freqs, magnitude=1.0):
    ang = np.outer(np.arange(first, first + positions, dtype=np.float64), freqs)
    return magnitude * np.concatenate([np.cos(ang), np.sin(ang)], 1)


def rope(x, cos_sin, neox):
    """x [..., R], cos_sin [..., R] (broadcast) -> rotated."""
    half = x.shape[-1] // 2
    c, s = cos_sin[..., :half], cos_sin[..., half:]
    a, b = (x[..., :half], x[..., half:]) if neox else (x[..., 0::2], x[..., 1::2])
    p, q = a * c - b * s, b * c + a * s
    return np.concatenate([p, q], -1) if neox else np.stack([p, q], -1).reshape(x.shape)


def gather_rows(block_table, starts, cu, page_size, tokens):
    """Cache slot of each output row, -1 for rows that no request owns."""
    slots = np.full(tokens, -1, dtype=np.int64)
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            tok = int(starts[b]) + i
            slots[cu[b] + i] = int(block_table[b][tok // page_size]) * page_size + tok % page_size
    return slots


def prefill(q, k, v, cu_q, cu_k, scale, causal):
    """q [Tq, H, D], k [Tk, H, D], v [Tk, H, E].  Returns out, lse, the same sum over
    |v| (what rounded weights are off by, in units of their step) and each row's
    largest sum of |q k| over its keys (what the scores are off by)."""
    tq, h, e = q.shape[0], q.shape[1], v.shape[2]
    out, mass = np.zeros((tq, h, e)), np.zeros((tq, h, e))
    lse, size = np.full((tq, h), -np.inf), np.zeros((tq, h))
    for b in range(len(cu_q) - 1):
        keys = slice(cu_k[b], cu_k[b + 1])
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(n):
            seen = m - n + 1 + i if causal else m
            if seen <= 0:
                continue
            row = cu_q[b] + i
            kk, vv = k[keys][:seen], v[keys][:seen]
            s = scale * np.einsum("hd,khd->hk", q[row], kk)
            top = s.max(1, keepdims=True)
            top = np.where(np.isneginf(top), 0.0, top)
            p = np.exp(s - top)
            total = p.sum(1)
            with np.errstate(divide="ignore", invalid="ignore"):
                w = np.where(total[:, None] == 0, 0.0, p / total[:, None])
                lse[row] = np.log(total) + top[:, 0]
                out[row] = np.einsum("hk,khe->he", w, vv)
                mass[row] = np.einsum("hk,khe->he", w, np.abs(vv))
            size[row] = scale * np.einsum("hd,khd->hk", np.abs(q[row]), np.abs(kk)).max(1)
    return out, lse, mass, size


def merge(out_a, lse_a, out_b, lse_b):
    with np.errstate(invalid="ignore", divide="ignore"):
        lse = np.logaddexp(lse_a, lse_b)
        wa = np.where(np.isneginf(lse_a), 0.0, np.exp(lse_a - lse))
        wb = np.where(np.isneginf(lse_b), 0.0, np.exp(lse_b - lse))
    pa, pb = (np.where(w[..., None] == 0, 0.0, w[..., None] * o) for w, o in ((wa, out_a), (wb, out_b)))
    return pa + pb, lse
