"""The prompt's operators on the GPU against the float64 oracle.

Tolerances.  A bf16 result is off by half a step (2^-8 of the value) from an fp32
value.  Attention: every weight enters the second product rounded to bf16, so the
sum is off by at most 2^-8 of the same sum over |v|; a score is a sum of 192 exact
products in at most 24 additions of the tensor core, each off by 2^-22 of the sum of
the magnitudes (a truncated one), and the softmax moves by twice that; the sum over
L keys adds L / 8 additions of 2^-22 of the sum over |v|."""

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


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(*shape, seed=0, dtype=BF, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * gain).to(dtype).cuda()


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# ---- attention


class Attn:
    def __init__(self, h, q_lens, k_lens, causal, seed=0, gain=2.0, apart=False):
        tq, tk = sum(q_lens), sum(k_lens)
        self.h, self.causal = h, causal
        q, kv = randn(tq, h, 192, seed=seed, gain=gain), randn(tk, h, 256, seed=seed + 1)
        self.q_nope, self.q_pe, self.k_nope, self.v = q[..., :128], q[..., 128:], kv[..., :128], kv[..., 128:]
        if apart:  # arrays of their own instead of slices
            self.q_nope, self.q_pe, self.k_nope, self.v = (x.contiguous() for x in (self.q_nope, self.q_pe, self.k_nope, self.v))
        self.k_pe = randn(tk, 64, seed=seed + 2)
        self.cu_q, self.cu_k = cu(q_lens), cu(k_lens)
        self.out = torch.full((tq, h, 128), 7.0, dtype=BF, device="cuda")
        self.lse = torch.full((tq, h), 7.0, device="cuda")
        need = B.mla_prefill_workspace_bytes(tq, tk, len(q_lens), h)
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None

    def run(self, scale=SCALE):
        B.mla_prefill(self.q_nope, self.q_pe, self.k_nope, self.k_pe, self.v, self.cu_q, self.cu_k, self.causal, scale,
                      self.out, self.lse, self.ws)
        return self.out, self.lse

    def oracle(self, scale=SCALE):
        k = np.concatenate([f64(self.k_nope), np.broadcast_to(f64(self.k_pe)[:, None], (self.k_pe.shape[0], self.h, 64))], 2)
        q = np.concatenate([f64(self.q_nope), f64(self.q_pe)], 2)
        return O.prefill(q, k, f64(self.v), self.cu_q.tolist(), self.cu_k.tolist(), scale, self.causal)

    def check(self, scale=SCALE, rows=slice(None)):
        want, want_lse, mass, size = self.oracle(scale)
        got, got_lse = f64(self.out), f64(self.lse)
        longest = int((self.cu_k[1:] - self.cu_k[:-1]).max())
        score = 24 * 2.0 ** -22 * size + 2.0 ** -20
        tol = (2.0 ** -8 + 2 * score[..., None] + longest / 8 * 2.0 ** -22) * mass + 2.0 ** -8 * np.abs(want) + 1e-30
        bad = ~(np.abs(got - want) <= tol)
        assert not bad[rows].any(), (np.argwhere(bad)[:4], np.abs(got - want)[rows].max())
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse)[rows], empty[rows]) and np.all(got[rows][empty[rows]] == 0)
        with np.errstate(invalid="ignore"):
            off = np.abs(got_lse - want_lse) - score - 2.0 ** -21 * np.abs(want_lse)
        assert not (off[rows][~empty[rows]] > 0).any(), np.nanmax(off)


CASES = [
    (1, [1], [1], True), (1, [1], [1], False), (2, [3], [3], True), (3, [128], [128], True), (1, [127], [129], True),
    (2, [129], [129], True), (1, [256], [256], True), (1, [257], [257], True), (2, [255], [700], True),
    (1, [640], [640], True), (2, [500], [500], False), (1, [1], [1000], True), (1, [1], [1000], False),
    (3, [5, 0, 300, 1], [5, 9, 300, 640], True), (2, [130, 64, 0, 1, 257], [0, 400, 0, 1, 511], False),
    (1, [300], [100], True), (2, [300, 7], [0, 7], True), (5, [40] * 40, [40] * 40, True), (1, [1] * 70, [300] * 70, True),
    # few rows and many keys: the keys are cut into parts
    (2, [100], [5000], False), (1, [1], [20000], True), (3, [600], [4000], True), (2, [5, 0, 300], [3000, 2500, 0], True),
    (2, [700, 3], [1100, 3500], True), (1, [40, 30, 1], [1500, 0, 9000], False),
    (16, [130], [130], True), (1, [513, 511], [513, 1025], True), (1, [2], [384], False), (1, [200], [256], False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"h{c[0]}-{'.'.join(map(str, c[1]))[:24]}-{'.'.join(map(str, c[2]))[:24]}-{c[3]}")
def test_attention(case):
    a = Attn(*case, seed=len(case[1]) + case[0])
    a.run()
    a.check()
    if case[0] == 2:
        b = Attn(*case, seed=len(case[1]) + case[0], apart=True)
        b.run()
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


# ---- rotary table and rotation

TABLES = [(0, 100, 64, "plain", 1.0, 1e4, 1.0), (0, 5000, 64, "yarn", 40.0, 1e4, 1.0), (131000, 333, 64, "linear", 8.0, 5e5, 1.25),
          ((1 << 31) - 64, 64, 32, "plain", 1.0, 1e4, 1.0), (7, 9, 2, "plain", 1.0, 1e4, 0.5), (3, 50, 40, "yarn", 2.5, 1e4, 1.1),
          (12345, 77, 30, "yarn", 16.0, 1e6, 1.0), (0, 3, 512, "plain", 1.0, 1e4, -2.0)]
SCALINGS = {"plain": B.MLA_ROPE_PLAIN, "linear": B.MLA_ROPE_LINEAR, "yarn": B.MLA_ROPE_YARN}


@pytest.mark.parametrize("first,n,dim,scaling,factor,base,magnitude", TABLES)
def test_rope_table(first, n, dim, scaling, factor, base, magnitude):
    t = torch.full((n, dim), 9.0, device="cuda")
    B.mla_rope_table(t, first, base, SCALINGS[scaling], factor, 4096, 32.0, 1.0, magnitude)
    want = O.rope_table(first, n, O.rope_frequencies(dim, base, scaling, factor), magnitude)
    # sincospif, the correction and the product: at most 4 units of 2^-24 of a number below 1; the oracle's own
    # angle in 64 bits: 2^-52 of itself
    tol = (4 * 2.0 ** -24 + 2.0 ** -52 * (first + n)) * abs(magnitude)
    assert np.abs(f64(t) - want).max() <= tol


def test_rope_table_rows_do_not_depend_on_the_window():
    a, b = torch.empty(1000, 64, device="cuda"), torch.empty(300, 64, device="cuda")
    B.mla_rope_table(a, 0)
    B.mla_rope_table(b, 700)
    assert torch.equal(a[700:], b)
    c = torch.empty(1000 * 64 + 1, device="cuda")[1:].view(1000, 64)  # rows off the 16-byte grid: the narrow form
    B.mla_rope_table(c, 0)
    assert torch.equal(a, c)


def rotated(x, cs, neox):
    """The formula with every product and sum rounded to fp32: bits to match."""
    half = x.shape[-1] // 2
    x, c, s = x.float(), cs[..., :half], cs[..., half:]
    a, b = (x[..., :half], x[..., half:]) if neox else (x[..., 0::2], x[..., 1::2])
    p, q = a * c - b * s, b * c + a * s
    return (torch.cat([p, q], -1) if neox else torch.stack([p, q], -1).flatten(-2)).to(BF)


@pytest.mark.parametrize("neox", [False, True])
@pytest.mark.parametrize("t,h,r", [(1, 1, 64), (5, 16, 64), (130, 128, 64), (33, 3, 40), (17, 7, 6), (9, 300, 64), (4, 2, 512), (300, 1, 2)])
def test_rope(t, h, r, neox):
    cs = torch.empty(500, r, device="cuda")
    B.mla_rope_table(cs)
    pos = torch.randint(0, 500, (t,), generator=torch.Generator().manual_seed(t)).cuda()
    q, k = randn(t, h, 128 + r, seed=1), randn(t, 512 + r, seed=2)
    q_out, k_out = torch.zeros(t, h, r, dtype=BF, device="cuda"), torch.zeros(t, r, dtype=BF, device="cuda")
    B.mla_rope(q[..., 128:], k[:, 512:], pos, cs, neox, q_out, k_out)
    assert torch.equal(q_out, rotated(q[..., 128:], cs[pos][:, None], neox))
    assert torch.equal(k_out, rotated(k[:, 512:], cs[pos], neox))
    want = O.rope(f64(q[..., 128:]), f64(cs)[pos.cpu().numpy()][:, None], neox)
    assert np.all(np.abs(f64(q_out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21)  # (a sum that cancels: 3 steps of 2^-23)
    # in place, alone, and off the 16-byte grid
    q2, k2 = q.clone(), k.clone()
    B.mla_rope(q2[..., 128:], None, pos, cs, neox, q2[..., 128:], None)
    B.mla_rope(None, k2[:, 512:], pos, cs, neox, None, k2[:, 512:])
    assert torch.equal(q2[..., 128:], q_out) and torch.equal(k2[:, 512:], k_out)
    assert torch.equal(q2[..., :128], q[..., :128]) and torch.equal(k2[:, :512], k[:, :512])
    odd = torch.zeros(t, h, r + 3, dtype=BF, device="cuda")
    B.mla_rope(q[..., 127:127 + r], None, pos, cs, neox, odd[..., 1:1 + r], None)
    assert torch.equal(odd[..., 1:1 + r], rotated(q[..., 127:127 + r], cs[pos][:, None], neox))
    assert not odd[..., 0].any() and not odd[..., 1 + r:].any()


def test_rope_positions_outside_the_table():
    cs = torch.empty(10, 64, device="cuda")
    B.mla_rope_table(cs)
    q, k = randn(4, 2, 64, seed=1), randn(4, 64, seed=2)
    q_out, k_out = torch.full_like(q, 5.0), torch.full_like(k, 5.0)
    B.mla_rope(q, k, torch.tensor([3, 10, -1, 9], device="cuda"), cs, True, q_out, k_out)
    assert B.mla_decode_device_error() == 0x801
    assert torch.all(q_out[1:3] == 5) and torch.all(k_out[1:3] == 5)
    assert torch.equal(q_out[[0, 3]], rotated(q[[0, 3]], cs[[3, 9]][:, None], True))


# ---- gather


@pytest.mark.parametrize("page", [32, 64])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("latent", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,starts", [([1], [0]), ([5, 0, 70, 1], [0, 3, 63, 200]), ([0, 0, 130], [9, 0, 1]),
                                         ([3] * 50, list(range(50))), ([1] * 1100, [7] * 1100)])
def test_gather(page, cache, latent, lens, starts):
    t, batch = sum(lens), len(lens)
    blocks = [-(-(a + n) // page) for a, n in zip(starts, lens)]
    width, pool = max(blocks) + 2, sum(blocks) + 2
    g = torch.Generator().manual_seed(t)
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table, at = torch.full((batch, width), -1, dtype=torch.int32), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    rows = torch.randn(pool, page, 576, generator=g) * 3
    rows[0, :, :128] = 0  # blocks of zeros
    kv = rows.to(F8 if cache == "e4m3" else BF).cuda()
    k_scale = 0.3 if cache == "e4m3" else 1.0
    pad = 3  # rows past the last request's
    lat = torch.zeros(t + pad, 512 + 16, dtype=F8 if latent == "e4m3" else BF, device="cuda")[:, :512]
    pe = torch.full((t + pad, 72), 9.0, dtype=BF, device="cuda")[:, :64]
    sc = torch.full((4, t + pad + 5), 9.0, device="cuda")[:, :t + pad] if latent == "e4m3" else None
    B.mla_cache_gather(kv, B.MLA_KV_E4M3 if cache == "e4m3" else B.MLA_KV_BF16, table.cuda(),
                       torch.tensor(starts, dtype=torch.int32, device="cuda"), cu(lens), k_scale, lat,
                       B.MLA_OUT_E4M3 if latent == "e4m3" else B.MLA_OUT_BF16, sc, pe)
    slots = torch.from_numpy(O.gather_rows(table.numpy(), starts, np.concatenate([[0], np.cumsum(lens)]), page, t)).cuda()
    src = kv.view(torch.uint8 if cache == "e4m3" else torch.int16).view(-1, 576)[slots].view(kv.dtype)
    assert torch.equal(pe[:t], (src[:, 512:].float() * torch.tensor(k_scale, device="cuda")).to(BF))
    if latent == "bf16":
        assert torch.equal(lat[:t], (src[:, :512].float() * torch.tensor(k_scale, device="cuda")).to(BF))
    elif cache == "e4m3":
        assert torch.equal(lat[:t].view(torch.uint8), src[:, :512].view(torch.uint8))
        assert torch.all(sc[:, :t] == torch.tensor(k_scale, device="cuda"))
    else:  # the library's own quantiser
        y, ys = torch.empty(t, 512, dtype=F8, device="cuda"), torch.empty(4, t, device="cuda")
        B.mla_act_quantize(src[:, :512].contiguous(), B.MLA_ACT_NONE, y, B.MLA_OUT_E4M3, ys)
        assert torch.equal(lat[:t].view(torch.uint8), y.view(torch.uint8)) and torch.equal(sc[:, :t], ys)
    assert not lat[t:].view(torch.uint8).any() and torch.all(pe[t:] == 9)
    assert sc is None or torch.all(sc[:, t:] == 9)


def test_gather_refuses_what_it_cannot_find():
    kv = torch.ones(4, 32, 576, dtype=BF, device="cuda")
    lat, pe = torch.zeros(40, 512, dtype=BF, device="cuda"), torch.zeros(40, 64, dtype=BF, device="cuda")

    def run(table, starts, lens):
        lat.zero_()
        pe.zero_()
        B.mla_cache_gather(kv, B.MLA_KV_BF16, torch.tensor(table, dtype=torch.int32, device="cuda"),
                           torch.tensor(starts, dtype=torch.int32, device="cuda"), lens, 1.0, lat, B.MLA_OUT_BF16, None, pe)
        done = (lat == 1).all(1) & (pe == 1).all(1)
        assert torch.equal(done, (lat != 0).any(1) | (pe != 0).any(1))  # whole rows or nothing
        return B.mla_decode_device_error(), done.nonzero()[:, 0].tolist()

    assert run([[0, 1]], [60], cu([8])) == (0x901, [0, 1, 2, 3])        # past the table's row
    assert run([[0, 1]], [-2], cu([4])) == (0x901, [2, 3])
    assert run([[0, 4]], [30], cu([4])) == (0x902, [0, 1])              # a page outside the pool
    assert run([[-1, 3]], [30], cu([4])) == (0x902, [2, 3])
    code, _ = run([[0, 1], [2, 3]], [0, 0], torch.tensor([0, 9, 5], dtype=torch.int32, device="cuda"))
    assert code == 0x903
    code, _ = run([[0, 1], [2, 3]], [0, 0], torch.tensor([-5, 9, 99], dtype=torch.int32, device="cuda"))
    assert code in (0x901, 0x903)                                       # (the first that was met)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_gather_quantises_what_is_not_finite(bad):
    """A block with a NaN is NaN, one with an infinity keeps its place; others are untouched."""
    kv = torch.ones(1, 32, 576, dtype=BF, device="cuda")
    kv[0, 3, 130] = bad
    lat, sc, pe = torch.zeros(8, 512, dtype=F8, device="cuda"), torch.zeros(4, 8, device="cuda"), torch.zeros(8, 64, dtype=BF, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    B.mla_cache_gather(kv, B.MLA_KV_BF16, table, None, cu([8]), 1.0, lat, B.MLA_OUT_E4M3, sc, pe)
    y, ys = torch.empty_like(lat), torch.empty_like(sc)
    B.mla_act_quantize(kv[0, :8, :512].contiguous(), B.MLA_ACT_NONE, y, B.MLA_OUT_E4M3, ys)
    assert torch.equal(lat.view(torch.uint8), y.view(torch.uint8)) and torch.equal(sc.isnan(), ys.isnan())
    assert torch.equal(sc.nan_to_num(1.0), ys.nan_to_num(1.0))


# ---- merge


@pytest.mark.parametrize("t,h,d", [(1, 1, 8), (1, 1, 128), (7, 3, 128), (5, 16, 512), (3, 5, 72), (2, 3, 2048), (300, 2, 128)])
def test_merge(t, h, d):
    a, b = randn(t, h, d + 8, seed=1)[..., :d], randn(h, t, d, seed=2).transpose(0, 1)
    la, lb = randn(t, h, seed=3, dtype=torch.float32, gain=3.0), randn(t, h, seed=4, dtype=torch.float32, gain=3.0)
    la[0, 0] = lb[-1, -1] = -float("inf")
    out, lse = torch.empty(t, h, d, dtype=BF, device="cuda"), torch.empty(t, h, device="cuda")
    B.mla_merge_states(a, la, b, lb, out, lse)
    want, want_lse = O.merge(f64(a), f64(la), f64(b), f64(lb))
    mass, _ = O.merge(np.abs(f64(a)), f64(la), np.abs(f64(b)), f64(lb))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(f64(lse)), empty) and not f64(out)[empty].any()
    # fp32: a weight is off by the exponent's rounding (2^-24 of up to 24) and a few steps; then half a bf16 step
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mass)
    assert np.all(np.abs(f64(lse) - want_lse)[~empty] <= 2.0 ** -20 * (1 + np.abs(want_lse)[~empty]))
    # into either part's own arrays
    for k in range(2):
        x, y, lx, ly = a.clone(), b.clone(), la.clone(), lb.clone()
        o, l = ((x, lx), (y, ly))[k]
        B.mla_merge_states(x, lx, y, ly, o, l)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_merge_of_parts_that_weigh_nothing():
    inf, nan = float("inf"), float("nan")
    a, b = torch.full((3, 1, 128), nan, dtype=BF, device="cuda"), torch.full((3, 1, 128), 2.0, dtype=BF, device="cuda")
    la = torch.tensor([[-inf], [-inf], [0.0]], device="cuda")
    lb = torch.tensor([[1.5], [-inf], [-inf]], device="cuda")
    out, lse = torch.empty_like(a), torch.empty_like(la)
    B.mla_merge_states(a, la, b, lb, out, lse)
    assert torch.all(out[0] == 2) and lse[0] == 1.5
    assert torch.all(out[1] == 0) and lse[1] == -inf
    assert out[2].isnan().all() and lse[2] == 0
    la[0], lb[0] = nan, 1.0
    B.mla_merge_states(a, la, b, lb, out, lse)
    assert lse[0].isnan() and out[0].isnan().all()


# ---- attention: masked places, offsets, strides


@pytest.mark.parametrize("h", [1, 3])
@pytest.mark.parametrize("q_lens,k_lens", [([40], [40]), ([300], [300]), ([700], [900]), ([5, 130, 260], [400, 130, 700]), ([90], [3000])])
@pytest.mark.parametrize("where", ["k_nope", "k_pe", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_may_hold_anything(h, q_lens, k_lens, where, bad):
    """A key or value that is not finite changes the rows that see it and no other."""
    a = Attn(h, q_lens, k_lens, True, seed=3)
    clean = [x.clone() for x in a.run()]
    x = getattr(a, where)
    ends = np.cumsum(k_lens)
    for end, n in zip(ends, q_lens):
        x[end - n // 2, ..., 5] = bad  # the second half of the request's rows see it
    a.run()
    row = 0
    for n in q_lens:
        first = n - n // 2
        assert torch.equal(a.out[row:row + first], clean[0][row:row + first])
        assert torch.equal(a.lse[row:row + first], clean[1][row:row + first])
        part = a.out[row + first:row + n].float()
        if where == "v":
            assert torch.equal(part[..., :5], clean[0][row + first:row + n, :, :5].float())
            assert torch.equal(part[..., 6:], clean[0][row + first:row + n, :, 6:].float())
            assert torch.equal(a.lse[row + first:row + n], clean[1][row + first:row + n])
            assert part[..., 5].isnan().all() if bad != bad else torch.all(part[..., 5] == bad)
        elif bad != bad:
            assert part.isnan().all() and a.lse[row + first:row + n].isnan().all()
        row += n


def test_values_of_both_infinities():
    a = Attn(2, [200], [200], True, seed=4)
    a.v[50, :, 7], a.v[150, :, 7] = float("inf"), -float("inf")
    a.run()
    col = a.out[:, :, 7].float()
    assert torch.all(col[:50].isfinite()) and torch.all(col[50:150] == float("inf")) and col[150:].isnan().all()


def test_rows_behind_the_last_key_and_rows_without_an_owner():
    """Rows past the last request, and the gaps that offsets leave, are not touched; keys there are not read."""
    a = Attn(2, [100, 50], [100, 50], True, seed=5)
    a.cu_q = torch.tensor([0, 60, 120], dtype=torch.int32, device="cuda")     # 30 rows at the end are no one's
    a.cu_k = torch.tensor([0, 60, 120], dtype=torch.int32, device="cuda")
    a.k_nope[120:], a.v[120:], a.k_pe[120:] = float("nan"), float("nan"), float("nan")
    a.run()
    assert torch.all(a.out[120:] == 7) and torch.all(a.lse[120:] == 7)
    a.k_nope[120:], a.v[120:], a.k_pe[120:] = 0, 0, 0
    a.check(rows=slice(0, 120))


@pytest.mark.parametrize("cq,ck,code,owned", [
    ([0, 30, 20, 60], [0, 30, 60, 90], 0xA01, [(0, 30)]),            # decreasing; then before an earlier one's end
    ([0, 30, 60, 500], [0, 30, 60, 90], 0xA01, [(0, 60)]),
    ([-5, 30, 60, 90], [0, 30, 60, 90], 0xA01, [(30, 90)]),
    ([0, 30, 60, 90], [0, 30, 20, 90], 0xA02, [(0, 30), (60, 90)]),
    ([0, 30, 60, 90], [0, 30, 60, 1000], 0xA02, [(0, 60)]),
    ([0, 30, 60, 90], [-1, 30, 60, 90], 0xA02, [(30, 90)]),
])
def test_offsets_that_break_the_rules(cq, ck, code, owned):
    a = Attn(2, [100], [100], False, seed=6)
    a.cu_q, a.cu_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cq, ck))
    a.run()
    assert B.mla_decode_device_error() == code
    done = torch.zeros(100, dtype=torch.bool, device="cuda")
    for lo, hi in owned:
        done[lo:hi] = True
    assert torch.equal((a.lse != 7).all(1), done) and torch.equal((a.out != 7).any(2).all(1), done)
    assert torch.equal((a.lse != 7).any(1), done)


def test_no_key_at_all():
    a = Attn(4, [5, 0, 300], [0, 0, 0], False)
    a.run()
    assert not a.out.any() and torch.all(a.lse == -float("inf"))


def test_scores_of_minus_infinity():
    a = Attn(1, [3], [200], False, seed=7)
    a.q_nope[1] = 0
    a.q_nope[1, :, 0] = 1
    a.k_nope[..., 0] = -float("inf")
    a.q_pe[1] = 0
    a.q_nope[0, :, 0], a.q_nope[2, :, 0] = 0, 0    # 0 times an infinity
    a.run()
    assert not a.out[1].any() and torch.all(a.lse[1] == -float("inf"))
    assert a.out[[0, 2]].isnan().all()


def test_large_scores():
    """Maxima that climb by far more than the running one is allowed to lag."""
    a = Attn(2, [300], [900], False, seed=8)
    step = torch.arange(900, device="cuda").float()
    a.q_nope[:], a.k_nope[:] = 0, 0
    a.q_nope[..., 0] = 16.0
    a.k_nope[..., 0] = (step[:, None] * 0.25).to(BF)
    a.run()
    a.check()
    a.k_nope[..., 0] = (step.flip(0)[:, None] * 0.25).to(BF)
    a.run()
    a.check()
    a.k_nope[..., 0] = torch.where(step[:, None] % 130 == 129, 300.0, -200.0).to(BF)
    a.run()
    a.check()


def test_strides():
    """Heads before tokens, wide gaps, a single head of many."""
    a = Attn(3, [70, 200], [70, 333], True, seed=9)
    want = [x.clone() for x in a.run()]
    gaps = lambda x, pad: torch.nn.functional.pad(x, (0, pad))[..., :x.shape[2]]  # noqa: E731
    a.q_nope, a.q_pe, a.k_nope = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (a.q_nope, a.q_pe, a.k_nope))
    a.v, a.k_pe = gaps(a.v, 24), torch.nn.functional.pad(a.k_pe, (0, 8))[:, :64]
    a.out = torch.full((3, 270, 136), 7.0, dtype=BF, device="cuda")[..., :128].transpose(0, 1)
    a.run()
    assert torch.equal(a.out, want[0]) and torch.equal(a.lse, want[1])
    for h in range(3):
        one = Attn(1, [70, 200], [70, 333], True, seed=9)
        one.q_nope, one.q_pe, one.k_nope, one.v = (x[:, h:h + 1] for x in (a.q_nope, a.q_pe, a.k_nope, a.v))
        one.k_pe = a.k_pe
        one.run()
        assert torch.equal(one.out, want[0][:, h:h + 1]) and torch.equal(one.lse, want[1][:, h:h + 1])


def test_workspace_is_asked_for():
    need = B.mla_prefill_workspace_bytes(100, 50000, 1, 2)
    assert need > 0
    a = Attn(2, [100], [50000], False)
    for ws in (None, a.ws[:need - 256], a.ws[128:]):
        with pytest.raises(B.MlaError) as e:
            B.mla_prefill(a.q_nope, a.q_pe, a.k_nope, a.k_pe, a.v, a.cu_q, a.cu_k, False, SCALE, a.out, a.lse, ws)
        assert e.value.code == B.MLA_ERR_WORKSPACE
    assert torch.all(a.out == 7)
