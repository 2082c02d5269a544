"""One FP8 decoder layer on a decode batch, from hidden states to hidden states,
in the library's calls: norm and quantisation, projections, rotation and cache
write, paged MLA decode, output projection, routed experts.

    python examples/fp8_layer_step.py            # needs a GPU; prints the error against plain torch

Weights are random.  ``LayerStep.run`` is what a serving loop does per step;
``LayerStep.plain`` repeats it in elementary torch operations (fp32, with the
same roundings to e4m3) and is only there to check the result.
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_mla_decode_08_gb300 import binding as B  # noqa: E402

LATENT, ROPE, PAGE, BLOCK = 512, 64, 64, 128
EPS = 1e-6


def quantized_weights(shape, gen):
    """Random e4m3 weights [..., n, k] with a scale for each 128 x 128 block (n, k multiples of 128)."""
    w = torch.randn(*shape, device="cuda", generator=gen) / math.sqrt(shape[-1])
    t = w.view(*shape[:-2], shape[-2] // BLOCK, BLOCK, shape[-1] // BLOCK, BLOCK)
    s = t.abs().amax((-3, -1)) / 448.0
    return (t / s[..., :, None, :, None]).reshape(shape).to(torch.float8_e4m3fn), s.contiguous()


class LayerStep:
    def __init__(self, batch=8, hidden=1024, heads=16, experts=8, top_k=2, ffn=512, max_len=640, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.hidden, self.heads, self.experts, self.top_k, self.ffn = batch, hidden, heads, experts, top_k, ffn
        self.scale = 1.0 / math.sqrt(192)
        rows = heads * (LATENT + ROPE) + LATENT + ROPE  # absorbed queries, then the latent row
        rows += -rows % BLOCK
        self.w_qkv = quantized_weights((rows, hidden), g)
        self.w_out = quantized_weights((hidden, heads * LATENT), g)
        self.w_router = quantized_weights((BLOCK, hidden), g)  # its first `experts` rows count
        self.w_up = quantized_weights((experts, 2 * ffn, hidden), g)
        self.w_down = quantized_weights((experts, hidden, ffn), g)
        self.norms = [(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16() for d in (hidden, LATENT, hidden)]
        # a cache that already holds every request's earlier tokens
        self.lens = torch.randint(1, max_len, (batch,), device="cuda", generator=g, dtype=torch.int32)
        blocks = -(-max_len // PAGE)
        self.table = torch.randperm(batch * blocks, device="cuda", generator=g).to(torch.int32).view(batch, blocks)
        self.cache = torch.randn(batch * blocks, PAGE, LATENT + ROPE, device="cuda", generator=g).to(torch.float8_e4m3fn)
        pos = (self.lens - 1).long()
        self.positions = pos
        self.slots = self.table.long().gather(1, (pos // PAGE)[:, None])[:, 0] * PAGE + pos % PAGE
        ang = torch.arange(max_len)[:, None] * 10000.0 ** (-torch.arange(0, ROPE, 2) / ROPE)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.plan = B.mla_decode_plan_device(batch, PAGE, heads)
        self.workspace = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def run(self, x, residual):
        """x bf16 [batch, hidden], residual bf16 (updated in place) -> bf16 [batch, hidden] and the routing used."""
        t, d, h, dev = self.batch, self.hidden, self.heads, "cuda"
        new8 = lambda rows, cols: torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=dev)  # noqa: E731
        new16 = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device=dev)  # noqa: E731
        scales = lambda rows, cols: torch.empty(-(-cols // BLOCK), rows, device=dev)  # noqa: E731

        # attention: norm, projection, rotation and cache write, decode, output projection
        y, ys = new8(t, d), scales(t, d)
        B.mla_add_rmsnorm(x, residual, residual, B.MLA_OUT_BF16, self.norms[0], EPS, y, B.MLA_OUT_E4M3, ys)
        qkv = new16(t, self.w_qkv[0].shape[0])
        B.mla_gemm_fp8(y, ys, *self.w_qkv, qkv, B.MLA_OUT_BF16)
        q = qkv[:, :h * (LATENT + ROPE)].view(t, h, LATENT + ROPE)
        kv = qkv[:, h * (LATENT + ROPE):][:, :LATENT + ROPE]
        k_nope = new16(t, LATENT)
        B.mla_add_rmsnorm(kv[:, :LATENT], None, None, 0, self.norms[1], EPS, k_nope, B.MLA_OUT_BF16)
        q8 = torch.empty(t, h, LATENT + ROPE, dtype=torch.float8_e4m3fn, device=dev)
        B.mla_rope_quantize_cache_write(q[..., :LATENT].contiguous(), q[..., LATENT:].contiguous(), q8, B.MLA_Q_E4M3,
                                        k_nope, kv[:, LATENT:].contiguous(), self.positions, self.cos_sin, False,
                                        self.cache, B.MLA_KV_E4M3, self.slots)
        attn, lse = new16(t, h, LATENT), torch.empty(t, h, device=dev)
        B.mla_decode_fp8q(self.plan, q8, self.cache, self.table, self.lens, self.scale, 1.0, attn, lse, self.workspace)
        o, os_ = new8(t, h * LATENT), scales(t, h * LATENT)
        B.mla_act_quantize(attn.view(t, h * LATENT), B.MLA_ACT_NONE, o, B.MLA_OUT_E4M3, os_)
        mixed = new16(t, d)
        B.mla_gemm_fp8(o, os_, *self.w_out, mixed, B.MLA_OUT_BF16)

        # experts: norm, router (fp32 results), rows sorted by expert, gated unit between two grouped products
        B.mla_add_rmsnorm(mixed, residual, residual, B.MLA_OUT_BF16, self.norms[2], EPS, y, B.MLA_OUT_E4M3, ys)
        logits = torch.empty(t, BLOCK, device=dev)
        B.mla_gemm_fp8(y, ys, *self.w_router, logits, B.MLA_OUT_FP32)
        gate, expert = torch.softmax(logits[:, :self.experts], 1).topk(self.top_k)
        order = expert.flatten().argsort(stable=True)
        rows = order // self.top_k
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=dev)
        offsets[1:] = torch.bincount(expert.flatten(), minlength=self.experts).cumsum(0)
        n = t * self.top_k
        up = new16(n, 2 * self.ffn)
        B.mla_grouped_gemm_fp8(y.view(torch.uint8)[rows], ys[:, rows].contiguous(), *self.w_up, offsets, up, B.MLA_OUT_BF16)
        f, fs = new8(n, self.ffn), scales(n, self.ffn)
        B.mla_act_quantize(up, B.MLA_ACT_SILU_MUL, f, B.MLA_OUT_E4M3, fs)
        down = new16(n, d)
        B.mla_grouped_gemm_fp8(f, fs, *self.w_down, offsets, down, B.MLA_OUT_BF16)
        out = torch.zeros(t, d, device=dev)
        out.index_add_(0, rows, down.float() * gate.flatten()[order][:, None])
        return out.bfloat16(), expert

    # ---- the same in plain torch

    @staticmethod
    def _weights(w):
        return w[0].float() * w[1].repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)

    @staticmethod
    def _rounded(v):
        """fp32 rows through e4m3 with a scale for each 128 columns."""
        b = v.view(v.shape[0], -1, BLOCK)
        s = b.abs().amax(2, keepdim=True).clamp_min(1e-10) / 448.0
        return ((b / s).to(torch.float8_e4m3fn).float() * s).view(v.shape)

    @staticmethod
    def _norm(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w.float()

    def _rotated(self, v):
        c, s = self.cos_sin[self.positions, :ROPE // 2], self.cos_sin[self.positions, ROPE // 2:]
        c, s = (c[:, None], s[:, None]) if v.dim() == 3 else (c, s)
        a, b = v[..., 0::2], v[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)

    def plain(self, x, residual, cache, expert):
        t, h = self.batch, self.heads
        res = x.float() + residual.float()
        y = self._rounded(self._norm(res, self.norms[0]))
        res = res.bfloat16().float()
        qkv = (y @ self._weights(self.w_qkv).t()).bfloat16().float()
        q = qkv[:, :h * (LATENT + ROPE)].view(t, h, LATENT + ROPE)
        kv = qkv[:, h * (LATENT + ROPE):][:, :LATENT + ROPE]
        e4m3 = lambda v: v.clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
        q = torch.cat([e4m3(q[..., :LATENT]), e4m3(self._rotated(q[..., LATENT:]))], -1).float()
        k_nope = self._norm(kv[:, :LATENT], self.norms[1]).bfloat16().float()
        cache = cache.clone()
        cache.view(-1, LATENT + ROPE)[self.slots] = torch.cat([e4m3(k_nope), e4m3(self._rotated(kv[:, LATENT:]))], -1)
        attn = torch.empty(t, h, LATENT, device="cuda")
        for b in range(t):
            keys = cache[self.table[b].long()].flatten(0, 1)[:self.lens[b]].float()
            attn[b] = torch.softmax(self.scale * (q[b] @ keys.t()), 1) @ keys[:, :LATENT]
        mixed = (self._rounded(attn.bfloat16().float().view(t, -1)) @ self._weights(self.w_out).t()).bfloat16().float()
        res = mixed + res
        y = self._rounded(self._norm(res, self.norms[2]))
        gate = torch.softmax((y @ self._weights(self.w_router).t())[:, :self.experts], 1).gather(1, expert)
        w_up, w_down = self._weights(self.w_up), self._weights(self.w_down)
        out = torch.zeros_like(y)
        for k in range(self.top_k):
            up = torch.einsum("td,tfd->tf", y, w_up[expert[:, k]]).bfloat16().float()
            f = self._rounded(torch.nn.functional.silu(up[:, :self.ffn]) * up[:, self.ffn:])
            out += gate[:, k, None] * torch.einsum("tf,tdf->td", f, w_down[expert[:, k]]).bfloat16().float()
        return out, res.bfloat16()


def main():
    step = LayerStep()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(step.batch, step.hidden, device="cuda", generator=g).bfloat16()
    residual = torch.randn(step.batch, step.hidden, device="cuda", generator=g).bfloat16()
    before, cache = residual.clone(), step.cache.clone()
    out, expert = step.run(x, residual)
    want, want_residual = step.plain(x, before, cache, expert)
    assert B.mla_decode_device_error() == 0
    rel = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    errors = rel(out, want), rel(residual, want_residual)
    print(f"layer step of {step.batch} tokens: relative error {errors[0]:.2e} (residual {errors[1]:.2e})")
    return errors


if __name__ == "__main__":
    main()
