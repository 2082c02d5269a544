"""The prompt's operators together, as a serving step uses them: in one run against the
absorbed decode, in graphs, on several streams, past 32-bit offsets."""

import numpy as np
import pytest
import torch

from oracle import prompt_ref as O
from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
SCALE = 1 / np.sqrt(192)


@pytest.fixture(autouse=True)
def no_device_error():
    B.mla_decode_device_error(reset=True)
    yield
    assert B.mla_decode_device_error(reset=True) == 0


def randn(*shape, seed=0, gain=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * gain).to(BF).cuda()


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def new(*shape):
    return torch.empty(*shape, dtype=BF, device="cuda")


def prefill(q_nope, q_pe, k_nope, k_pe, v, cq, ck, causal, out, lse):
    need = B.mla_prefill_workspace_bytes(q_nope.shape[0], k_nope.shape[0], cq.numel() - 1, q_nope.shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    B.mla_prefill(q_nope, q_pe, k_nope, k_pe, v, cq, ck, causal, SCALE, out, lse, ws)


@pytest.mark.parametrize("chunk", [4096, 70])
def test_prompt_step_equals_the_absorbed_decode(chunk):
    """New tokens behind cached prefixes: rotation, cache write, prefixes gathered and
    expanded in chunks, attention over them and over the new tokens, merged; against the
    decode of the same tokens over the same cache with absorbed weights.

    Tolerance: the sides differ by roundings to bf16 at different places, each off by at
    most 2^-8 of a value and by 2^-8 / sqrt(3) as a standard deviation at the most.  Keys,
    values and latent rows have a deviation of 1, queries one of 2, so the keys' roundings
    move a score by scale * 2 * sqrt(128) * 2^-8 / sqrt(3) = 0.004 and those of the absorbed
    query (deviation 1) by scale * sqrt(512) * 2^-8 / sqrt(3) = 0.004; the weights' and the
    values' roundings are 2^-8 of a term.  Together below 0.01 of a result's size and of
    an lse; five times that is allowed for the rows of few keys, sixteen for the largest
    of the lse's differences.  A wrong row, position or weight is off by a result's size.
    """
    h, page, lens, new_lens = 4, 64, [200, 33, 0, 129], [5, 32, 17, 1]
    total = sum(new_lens)
    w_k, w_v = randn(h, 128, 512, seed=1, gain=512 ** -0.5), randn(h, 128, 512, seed=2, gain=512 ** -0.5)
    table = torch.empty(1000, 64, device="cuda")
    B.mla_rope_table(table, 0, 1e4, B.MLA_ROPE_YARN, 4.0, 256)
    ends = [a + n for a, n in zip(lens, new_lens)]
    blocks = [-(-e // page) for e in ends]
    bt, at = torch.zeros(4, max(blocks), dtype=torch.int32), 0
    for b, n in enumerate(blocks):
        bt[b, :n] = torch.arange(at, at + n).flip(0)
        at += n
    cache, bt = randn(at, page, 576, seed=3), bt.cuda()
    position = torch.cat([torch.arange(a, e) for a, e in zip(lens, ends)])
    owner = torch.cat([torch.full((n,), b) for b, n in enumerate(new_lens)])
    slots = (bt.cpu()[owner, position // page].long() * page + position % page).cuda()
    position = position.cuda()

    # the step's projections, rotation and cache write
    q, kv = randn(total, h, 192, seed=4, gain=2.0), randn(total, 576, seed=5)
    q_pe, k_pe = new(total, h, 64), new(total, 64)
    B.mla_rope(q[..., 128:], kv[:, 512:], position, table, False, q_pe, k_pe)
    latent = kv[:, :512].contiguous()
    B.mla_rope_quantize_cache_write(None, None, None, B.MLA_Q_BF16, latent, kv[:, 512:].contiguous(), position, table, False,
                                    cache, B.MLA_KV_BF16, slots)
    assert torch.equal(cache.view(-1, 576)[slots], torch.cat([latent, k_pe], 1))  # both rotate to the same bits

    def expand(rows):  # a product of the caller's
        k = torch.einsum("tc,hdc->thd", rows.float(), w_k.float()).to(BF)
        return k, torch.einsum("tc,hdc->thd", rows.float(), w_v.float()).to(BF)

    cq = cu(new_lens)
    k, v = expand(latent)
    out, lse = new(total, h, 128), torch.empty(total, h, device="cuda")
    prefill(q[..., :128], q_pe, k, k_pe, v, cq, cq, True, out, lse)
    part, part_lse = torch.empty_like(out), torch.empty_like(lse)
    for start in range(0, max(lens), chunk):
        count = [min(chunk, max(0, n - start)) for n in lens]
        ck = cu(count)
        rows, pe = new(sum(count), 512), new(sum(count), 64)
        B.mla_cache_gather(cache, B.MLA_KV_BF16, bt, torch.full((4,), start, dtype=torch.int32, device="cuda"), ck, 1.0, rows,
                           B.MLA_OUT_BF16, None, pe)
        k, v = expand(rows)
        prefill(q[..., :128], q_pe, k, pe, v, cq, ck, False, part, part_lse)
        B.mla_merge_states(out, lse, part, part_lse, out, lse)

    # the absorbed form
    q_abs = torch.einsum("thd,hdc->thc", q[..., :128].float(), w_k.float()).to(BF).contiguous()
    plan = B.mla_decode_plan_ragged(ends, new_lens, page, h)
    ws = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    absorbed, want_lse = new(total, h, 512), torch.empty(total, h, device="cuda")
    B.mla_decode_ragged(plan, q_abs, q_pe, cache, B.MLA_KV_BF16, bt, torch.tensor(ends, dtype=torch.int32, device="cuda"), cq,
                        SCALE, 1.0, absorbed, want_lse, ws)
    want = torch.einsum("thc,hdc->thd", absorbed.float(), w_v.float())
    rel = float((out.float() - want).norm() / want.norm())
    assert rel <= 0.05 and float((lse - want_lse).abs().max()) <= 0.16, rel


def test_fp8_prefix_through_the_fp8_product():
    """Cached e4m3 rows, gathered as codes, are the FP8 product's operand as they are."""
    kv = (torch.randn(5, 64, 576, generator=torch.Generator().manual_seed(1)) * 2).to(F8).cuda()
    bt = torch.tensor([[3, 0, 4]], dtype=torch.int32, device="cuda")
    rows, sc, pe = torch.empty(150, 512, dtype=F8, device="cuda"), torch.empty(4, 150, device="cuda"), new(150, 64)
    B.mla_cache_gather(kv, B.MLA_KV_E4M3, bt, None, cu([150]), 0.25, rows, B.MLA_OUT_E4M3, sc, pe)
    w = torch.randn(256, 512, generator=torch.Generator().manual_seed(2)).to(F8).cuda()
    sw = torch.rand(2, 4, device="cuda")
    out = torch.empty(150, 256, device="cuda")
    B.mla_gemm_fp8(rows, sc, w, sw, out, B.MLA_OUT_FP32)
    src = kv[[3, 0, 4]].flatten(0, 1)[:150, :512].double() * 0.25
    wd = w.double() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    want, size = src @ wd.T, src.abs() @ wd.abs().T
    assert torch.all((out.double() - want).abs() <= 2.0 ** -18 * size)  # fp32 sums of 512 terms


class Step:
    """A captured step's buffers: rotation, gather, attention over both, merge."""

    def __init__(self, h, most_q, most_k, batch, seed):
        self.h, self.batch = h, batch
        self.q, self.kv = randn(most_q, h, 192, seed=seed), randn(most_k, h, 256, seed=seed + 1)
        self.k_raw, self.pos = randn(most_q, 64, seed=seed + 2), torch.arange(most_q, device="cuda") % 500
        self.cache = randn(most_k // 64 + batch, 64, 576, seed=seed + 3)
        self.bt = torch.arange(self.cache.shape[0], dtype=torch.int32, device="cuda").repeat(batch, 1)
        self.table = torch.zeros(500, 64, device="cuda")
        self.q_pe, self.k_pe = new(most_q, h, 64), new(most_q, 64)
        self.rows, self.pe = new(most_k, 512), new(most_k, 64)
        self.cq, self.ck = cu([0] * batch), cu([0] * batch)
        self.sources = [torch.zeros_like(self.cq), torch.zeros_like(self.ck)]
        self.outs = [torch.zeros(most_q, h, 128, dtype=BF, device="cuda") for _ in range(3)]
        self.lses = [torch.zeros(most_q, h, device="cuda") for _ in range(3)]
        self.ws = [torch.empty(max(256, B.mla_prefill_workspace_bytes(most_q, k, batch, h)), dtype=torch.uint8, device="cuda")
                   for k in (most_q, most_k)]

    def lengths(self, q_lens, k_lens):
        for s, lens in zip(self.sources, (q_lens, k_lens)):
            s.copy_(cu(lens))

    def run(self):
        self.cq.copy_(self.sources[0])
        self.ck.copy_(self.sources[1])
        B.mla_rope_table(self.table)
        B.mla_rope(self.q[..., 128:], self.k_raw, self.pos, self.table, False, self.q_pe, self.k_pe)
        B.mla_cache_gather(self.cache, B.MLA_KV_BF16, self.bt, None, self.ck, 1.0, self.rows, B.MLA_OUT_BF16, None, self.pe)
        n = self.q.shape[0]
        B.mla_prefill(self.q[..., :128], self.q_pe, self.kv[:n, :, :128], self.k_pe, self.kv[:n, :, 128:], self.cq, self.cq, True,
                      SCALE, self.outs[0], self.lses[0], self.ws[0])
        self.outs[1].zero_()
        B.mla_prefill(self.q[..., :128], self.q_pe, self.kv[..., :128], self.pe, self.kv[..., 128:], self.cq, self.ck, False, SCALE,
                      self.outs[1], self.lses[1], self.ws[1])
        B.mla_merge_states(self.outs[0], self.lses[0], self.outs[1], self.lses[1], self.outs[2], self.lses[2])

    def results(self):
        return [x.clone() for x in (*self.outs, *self.lses, self.rows, self.pe, self.q_pe)]

    def clear(self):
        for x in (*self.outs, *self.lses, self.rows, self.pe, self.q_pe, self.table):
            x.fill_(3)


LENGTHS = [([3, 0, 500], [900, 2000, 7]), ([600, 1, 1], [0, 0, 3000]), ([0, 0, 0], [0, 0, 0]), ([1, 1, 1], [1, 1, 1])]


@pytest.mark.parametrize("h", [2, 40])
def test_replay_serves_any_lengths(h):
    s = Step(h, 640, 3008, 3, seed=h)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for lens in LENGTHS + LENGTHS[::-1]:
        s.lengths(*lens)
        s.clear()
        s.run()
        torch.cuda.synchronize()
        want = s.results()
        s.clear()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, s.results()))


def test_streams_at_once():
    """Steps on their own streams and buffers, and two captured ones, give what each gives alone."""
    steps = [Step(h, 640, 3008, 3, seed=h) for h in (2, 16, 40)]
    want = []
    for s, lens in zip(steps, LENGTHS):
        s.lengths(*lens)
        s.clear()
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
        s.clear()
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for s, stream in zip(steps, streams):
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run()
        graphs.append(graph)
    for use_graphs in (False, True):
        for s in steps:
            s.clear()
        torch.cuda.synchronize()
        for _ in range(5):
            for s, stream, graph in zip(steps, streams, graphs):
                with torch.cuda.stream(stream):
                    graph.replay() if use_graphs else s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(w, s.results()))


def test_a_stream_given_by_name():
    s = Step(2, 64, 64, 1, seed=1)
    s.lengths([64], [64])
    s.run()
    torch.cuda.synchronize()
    want = s.outs[0].clone()
    s.outs[0].fill_(3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    B.mla_prefill(s.q[..., :128], s.q_pe, s.kv[:64, :, :128], s.k_pe, s.kv[:64, :, 128:], s.cq, s.cq, True, SCALE, s.outs[0],
                  s.lses[0], s.ws[0], stream=side)
    side.synchronize()
    assert torch.equal(s.outs[0], want)


def exact_rows(q, k, v):
    """fp64 attention of a few rows over all keys: q [n, 192], k [m, 192], v [m, 128].

    What the tests below allow, in units of the weights' mass sum w |v|: 2^-8 for weights
    rounded to bf16 (half a step), and as much again for scores off by up to 2^-9 (a sum
    of 192 fp32 products is off by 24 roundings of 2^-22 of sum |q k| scale < 60, which is
    below 2^-11) and for fp32 sums; and 2^-8 of the result for its own rounding."""
    w = torch.softmax(SCALE * (q.double() @ k.double().T), 1)
    return w @ v.double(), w @ v.double().abs()


def test_keys_past_32_bits():
    """Elements of keys and values beyond 2^31 (a wide row pitch), and their parts' merge."""
    tk, pitch = 20000, 1 << 17
    big = torch.zeros(tk, pitch, dtype=BF, device="cuda")
    big[:, -256:] = randn(tk, 256, seed=1)
    k, v = big[:, None, -256:-128], big[:, None, -128:]
    q, k_pe = randn(70, 1, 192, seed=2), randn(tk, 64, seed=3)
    out, lse = new(70, 1, 128), torch.empty(70, 1, device="cuda")
    prefill(q[..., :128], q[..., 128:], k, k_pe, v, cu([70]), cu([tk]), False, out, lse)
    want, mass = exact_rows(q[:, 0], torch.cat([k[:, 0], k_pe], 1), v[:, 0])
    assert torch.all((out[:, 0].double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs())


def test_queries_and_results_past_32_bits():
    tq, pitch = 20000, 1 << 17
    big = torch.zeros(tq, pitch, dtype=BF, device="cuda")
    big[:, :192] = randn(tq, 192, seed=1)
    q = big[:, None, :192]
    out = big[:, None, -128:]
    kv, k_pe, lse = randn(100, 1, 256, seed=2), randn(100, 64, seed=3), torch.empty(tq, 1, device="cuda")
    prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu([tq - 90, 90]), cu([0, 100]), True, out, lse)
    assert not out[:tq - 90].any() and torch.all(lse[:tq - 90] == -float("inf"))
    for i in (0, 89):
        want, mass = exact_rows(q[tq - 90 + i], torch.cat([kv[:11 + i, 0, :128], k_pe[:11 + i]], 1), kv[:11 + i, 0, 128:])
        assert torch.all((out[tq - 90 + i].double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs())
    # the rotation and the merge of the same rows
    table = torch.empty(tq, 64, device="cuda")
    B.mla_rope_table(table)
    pos = torch.arange(tq, device="cuda")
    small = new(tq, 1, 64)
    B.mla_rope(q[..., 128:], None, pos, table, True, small, None)
    B.mla_rope(q[..., 128:], None, pos, table, True, big[:, None, 1024:1088], None)
    assert torch.equal(small, big[:, None, 1024:1088])
    B.mla_merge_states(out, lse, out, lse, big[:, None, 2048:2176], torch.empty_like(lse))
    assert torch.equal(big[tq - 90:, None, 2048:2176], out[tq - 90:])


def test_a_cache_past_32_bits():
    pages = 40000  # of 64 rows of 1152 bytes: 2.9 GB
    kv = torch.zeros(pages, 64, 576, dtype=BF, device="cuda")
    kv[-1] = randn(64, 576, seed=1)
    bt = torch.full((1, 2), pages - 1, dtype=torch.int32, device="cuda")
    rows, pe = new(128, 512), new(128, 64)
    B.mla_cache_gather(kv, B.MLA_KV_BF16, bt, None, cu([128]), 1.0, rows, B.MLA_OUT_BF16, None, pe)
    assert torch.equal(rows, kv[-1, :, :512].repeat(2, 1)) and torch.equal(pe, kv[-1, :, 512:].repeat(2, 1))


def lens_of(batch, active, seed, most):
    g = np.random.default_rng(seed)
    lens = np.zeros(batch, dtype=int)
    lens[g.choice(batch, active, replace=False)] = g.integers(1, most + 1, active)
    return lens


@pytest.mark.parametrize("batch, active, most, h", [(500, 3, 700, 16), (300, 290, 5, 16), (129, 40, 300, 24), (4097, 2, 9, 2)])
def test_batches_padded_with_empty_requests(batch, active, most, h):
    """Every row of every request, wherever it lies among empty ones, whether clusters
    find one item, several or none."""
    lens = lens_of(batch, active, 1, most)
    extra = np.random.default_rng(2).integers(0, 200, batch) * (lens > 0)  # keys ahead of the new ones
    t, tk = int(lens.sum()), int((lens + extra).sum())
    q, kv, k_pe = randn(t + 3, h, 192, seed=1), randn(tk, h, 256, seed=2), randn(tk, 64, seed=3)
    out, lse = torch.full((t + 3, h, 128), 7, dtype=BF, device="cuda"), torch.full((t + 3, h), 7.0, device="cuda")
    prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu(lens), cu(lens + extra), True, out, lse)
    k = torch.cat([kv[..., :128], k_pe[:, None].expand(-1, h, -1)], -1).double()
    q0 = k0 = 0
    for n, m in zip(lens, lens + extra):
        if n:
            s = SCALE * torch.einsum("qhd,khd->hqk", q[q0:q0 + n].double(), k[k0:k0 + m])
            s.masked_fill_(torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None], -float("inf"))
            w, v = torch.softmax(s, -1), kv[k0:k0 + m, :, 128:].double()
            want, mass = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
            assert torch.all((out[q0:q0 + n].double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs())
            assert torch.all((lse[q0:q0 + n].double() - torch.logsumexp(s, -1).T).abs() <= 1e-4)
        q0, k0 = q0 + n, k0 + m
    assert torch.all(out[t:] == 7) and torch.all(lse[t:] == 7)


def test_gather_among_empty_requests():
    lens = lens_of(500, 30, 4, 3)
    t = int(lens.sum())
    kv = randn(70, 64, 576, seed=1)
    bt = torch.randint(0, 70, (500, 2), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    starts = torch.randint(0, 120, (500,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    rows, pe = torch.full((t + 5, 512), 7, dtype=BF, device="cuda"), torch.full((t + 5, 64), 7, dtype=BF, device="cuda")
    B.mla_cache_gather(kv, B.MLA_KV_BF16, bt, starts, cu(lens), 1.0, rows, B.MLA_OUT_BF16, None, pe)
    owner = torch.repeat_interleave(torch.arange(500), torch.tensor(lens)).cuda()
    token = starts[owner] + torch.tensor(np.concatenate([np.arange(n) for n in lens])).cuda()
    want = kv[bt[owner, token // 64].long(), token % 64]
    assert torch.equal(rows[:t], want[:, :512]) and torch.equal(pe[:t], want[:, 512:])
    assert torch.all(rows[t:] == 7) and torch.all(pe[t:] == 7)


def test_an_infinity_in_a_part_of_little_weight():
    """Its part weighs less than fp32 holds, but something: the row does not look finite."""
    a, b = torch.ones(1, 1, 8, dtype=BF, device="cuda"), torch.ones(1, 1, 8, dtype=BF, device="cuda")
    b[0, 0, 3] = float("inf")
    la, lb, out, lse = (torch.full((1, 1), x, device="cuda") for x in (0.0, -200.0, 0.0, 0.0))
    B.mla_merge_states(a, la, b, lb, out := new(1, 1, 8), lse)
    assert torch.isfinite(out).flatten().tolist() == [True] * 3 + [False] + [True] * 4 and float(lse) == 0.0
    # within one call, whose keys are cut into parts
    n = 20000
    q, k, k_pe, v = new(1, 1, 192).fill_(1), new(n, 1, 128).fill_(-8), new(n, 64).fill_(0), new(n, 1, 128).fill_(1)
    k[0] = 8
    v[n - 1, 0, 5] = float("inf")
    out, lse = new(1, 1, 128), torch.empty(1, 1, device="cuda")
    prefill(q[..., :128], q[..., 128:], k, k_pe, v, cu([1]), cu([n]), False, out, lse)
    assert not torch.isfinite(out[0, 0, 5]) and torch.all(out[0, 0, :5] == 1) and torch.all(out[0, 0, 6:] == 1)


def test_many_heads():
    t, h = 3, 2999
    q, kv, k_pe = randn(t, h, 192, seed=1), randn(t, h, 256, seed=2), randn(t, 64, seed=3)
    out, lse = new(t, h, 128), torch.empty(t, h, device="cuda")
    prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu([t]), cu([t]), True, out, lse)
    k = torch.cat([kv[..., :128], k_pe[:, None].expand(-1, h, -1)], -1).double()
    s = SCALE * torch.einsum("qhd,khd->hqk", q.double(), k)
    s.masked_fill_(torch.ones(t, t, dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    w, v = torch.softmax(s, -1), kv[..., 128:].double()
    want, mass = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
    assert torch.all((out.double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs())
    assert torch.equal(out[0], kv[0, :, 128:])  # one key


def test_offsets_that_begin_behind_the_first_row():
    """Rows ahead of the first request's and behind the last one's belong to no one."""
    q, kv, k_pe = randn(50, 2, 192, seed=1), randn(80, 2, 256, seed=2), randn(80, 64, seed=3)
    kv[:9], kv[70:], k_pe[:9], k_pe[70:], q[:11], q[40:] = (float("nan"),) * 6
    out, lse = torch.full((50, 2, 128), 7, dtype=BF, device="cuda"), torch.full((50, 2), 7.0, device="cuda")
    prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu([20, 9]) + 11, cu([50, 11]) + 9, True, out, lse)
    alone, alone_lse = new(29, 2, 128), torch.empty(29, 2, device="cuda")
    prefill(q[11:40, :, :128], q[11:40, :, 128:], kv[9:70, :, :128], k_pe[9:70], kv[9:70, :, 128:], cu([20, 9]), cu([50, 11]),
            True, alone, alone_lse)
    assert torch.equal(out[11:40], alone) and torch.equal(lse[11:40], alone_lse) and torch.isfinite(alone).all()
    assert torch.all(out[:11] == 7) and torch.all(out[40:] == 7) and torch.all(lse[:11] == 7) and torch.all(lse[40:] == 7)
    pages = randn(3, 64, 576, seed=4)
    rows, pe = torch.full((20, 512), 7, dtype=BF, device="cuda"), torch.full((20, 64), 7, dtype=BF, device="cuda")
    bt = torch.tensor([[2], [2]], dtype=torch.int32, device="cuda")  # a page of two requests
    B.mla_cache_gather(pages, B.MLA_KV_BF16, bt, None, cu([5, 7]) + 4, 1.0, rows, B.MLA_OUT_BF16, None, pe)
    assert torch.equal(rows[4:9], pages[2, :5, :512]) and torch.equal(rows[9:16], pages[2, :7, :512])
    assert torch.all(rows[:4] == 7) and torch.all(rows[16:] == 7) and torch.all(pe[:4] == 7) and torch.all(pe[16:] == 7)


@pytest.mark.parametrize("h, lens, ahead", [(3, [64, 5, 0, 64], [436, 0, 9, 7936]), (16, [1, 1, 1], [300, 9000, 300]), (2, [700, 3, 40], [5000, 100, 0]),
                                            (1, [2] * 31 + [1], [40] * 31 + [6000])])
def test_one_long_request_among_short_ones(h, lens, ahead):
    """Its keys are cut, theirs are not; an infinity reaches the rows that see it."""
    q, kv = randn(sum(lens), h, 192, seed=1), randn(sum(lens) + sum(ahead), h, 256, seed=2)
    k_pe = randn(kv.shape[0], 64, seed=3)
    keys = [a + n for a, n in zip(ahead, lens)]
    out, lse = new(sum(lens), h, 128), torch.empty(sum(lens), h, device="cuda")
    prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu(lens), cu(keys), True, out, lse)
    k = torch.cat([kv[..., :128], k_pe[:, None].expand(-1, h, -1)], -1).double()
    q0 = k0 = 0
    for n, m in zip(lens, keys):
        s = SCALE * torch.einsum("qhd,khd->hqk", q[q0:q0 + n].double(), k[k0:k0 + m])
        s.masked_fill_(torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None], -float("inf"))
        w, v = torch.softmax(s, -1), kv[k0:k0 + m, :, 128:].double()
        want, mass = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
        assert torch.all((out[q0:q0 + n].double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs())
        assert torch.all((lse[q0:q0 + n].double() - torch.logsumexp(s, -1).T).abs() <= 1e-4)
        q0, k0 = q0 + n, k0 + m
    again, again_lse = torch.empty_like(out), torch.empty_like(lse)
    kv[-1, :, 130] = float("inf")  # the last request's last key: seen by its last row
    prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cu(lens), cu(keys), True, again, again_lse)
    bad = torch.zeros_like(out, dtype=torch.bool)
    if lens[-1]:
        bad[-1, :, 2] = True
    assert torch.equal(~torch.isfinite(again), bad) and torch.equal(again[~bad], out[~bad]) and torch.equal(again_lse, lse)


def test_calls_in_a_row_share_a_workspace_and_feed_each_other():
    """Each call begins where the one before it ends: it reads that one's results, and
    replaces what it left in the workspace."""
    h, n = 4, 6000
    q, kv, k_pe = randn(64, h, 192, seed=1), randn(n, h, 256, seed=2), randn(n, 64, seed=3)
    need = max(B.mla_prefill_workspace_bytes(64, n, 1, h), B.mla_prefill_workspace_bytes(64, n, 2, h))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def steps(wait):
        x, outs = q.clone(), []
        for i in range(6):
            out, lse = new(64, h, 128), torch.empty(64, h, device="cuda")
            cq, ck = (cu([64]), cu([n])) if i % 2 else (cu([30, 34]), cu([n - 1000, 1000]))
            B.mla_prefill(x[..., :128], x[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cq, ck, False, SCALE, out, lse, ws)
            if wait:
                torch.cuda.synchronize()
            x = torch.cat([out, q[..., 128:]], -1) if i % 3 == 2 else x
            B.mla_merge_states(out, lse, out, lse, x[..., :128], torch.empty_like(lse))
            if wait:
                torch.cuda.synchronize()
            outs += [out, lse]
        return outs

    want = steps(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, steps(False)))
