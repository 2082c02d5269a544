"""GPU parity of the FP8 layer operators against the float64 oracle.

Tolerances, from the arithmetic:

* a code is within half a step of the value it stands for, 2^-4 relative or
  2^-10 of the scale for subnormal codes; with ``MLA_ACT_NONE`` the quantiser's
  float32 steps are repeated and codes and scales have to be equal;
* the norm's value carries the error of a sum of squares (at most 2^-20
  relative for the widths here), rsqrt (2 ulp) and three products: below 2^-18;
* the gated unit carries the fast exponential's 2 + 1.2 |g| ulp: below 2^-15
  for |g| <= 100;
* a product rounds once per 32-wide step (its 33 summands aligned to the largest
  with at least 25 bits kept: 33 * 2^-25 < 2^-19) and twice per block, below
  (k / 32 + blocks + 4) * 2^-19 of the sum of the terms' magnitudes, then half a
  step of its output type;
* with small integers and power-of-two scales every sum is exact in fp32, so
  the result has to equal the rounded exact value, bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_layer_ref as L
from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def no_device_error():
    B.mla_decode_device_error(reset=True)
    yield
    torch.cuda.synchronize()


def f64(t):
    return t.double().cpu().numpy()


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def outputs(t, d, y_dtype, stride=None):
    stride = stride or d
    kind = torch.float8_e4m3fn if y_dtype == B.MLA_OUT_E4M3 else torch.bfloat16
    y = torch.full((t, stride), 7.0, device="cuda").to(kind)
    sc = torch.full((L.blocks(d), t + 3), -5.0, device="cuda")
    return y, y[:, :d], sc, sc[:, :t]


def check_codes(y, sc, want, slack):
    s = f64(sc)
    amax = L.block_amax(want)
    assert np.all(np.abs(s * 448 - np.maximum(amax, 1e-10)) <= (slack + 2 * F32_HALF) * np.maximum(amax, 1e-10))
    spread = L.spread(s, want.shape[1])
    half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * spread)
    assert np.all(np.abs(f64(y) * spread - want) <= half * (1 + 16 * slack) + 16 * slack * np.abs(want))


# ------------------------------------------------------------------ rows


@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("y_dtype", [B.MLA_OUT_BF16, B.MLA_OUT_E4M3])
@pytest.mark.parametrize("t,d,pad", [(1, 1, 0), (3, 7, 2), (5, 128, 0), (128, 512, 64), (2, 1000, 0), (7, 1001, 7),
                                     (33, 4096, 0), (2, 8200, 8), (3, 16385, 0), (2, 32768, 0), (1, 32767, 1)])
def test_norm(t, d, pad, y_dtype, residual):
    rng = np.random.default_rng(t * 7919 + d)
    x = bf16(rng, (t, d + pad), 3.0)[:, :d]
    w = bf16(rng, (d,))
    res = None if residual is None else (torch.randn(t, d + pad, generator=torch.Generator().manual_seed(d))).to(residual).cuda()[:, :d]
    out = None if res is None else torch.zeros(t, d + pad, dtype=residual, device="cuda")[:, :d]
    yw, y, scw, sc = outputs(t, d, y_dtype, d + pad)
    B.mla_add_rmsnorm(x, res, out, B.MLA_OUT_FP32 if residual == torch.float32 else B.MLA_OUT_BF16, w, 1e-5, y, y_dtype,
                      sc if y_dtype == B.MLA_OUT_E4M3 else None)
    want, h = L.rmsnorm(f64(x), f64(w), np.float32(1e-5), None if res is None else f64(res))
    if res is not None:
        assert torch.equal(out, (x.float() + res.float()).to(residual))  # one fp32 sum, one rounding
    if y_dtype == B.MLA_OUT_BF16:
        assert np.all(np.abs(f64(y) - want) <= np.abs(want) * (BF16_HALF + 2.0 ** -17))
    else:
        check_codes(y, sc, want, 2.0 ** -18)
        assert torch.all(scw[:, t:] == -5)
    assert torch.all(yw[:, d:].float() == 7)


@pytest.mark.parametrize("t,d,pad", [(700, 2048, 0), (613, 1544, 8), (1300, 8192, 0), (900, 1032, 16), (640, 700, 0),
                                     (1000, 130, 0)])
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("y_dtype", [B.MLA_OUT_BF16, B.MLA_OUT_E4M3])
def test_norm_many_rows(t, d, pad, residual, y_dtype):
    """More rows than CTAs run at once: every row's own statistics, none left out."""
    test_norm(t, d, pad, y_dtype, residual)


def test_norm_many_rows_keep_apart():
    """A NaN row among many leaves the rows before and after it (same CTA) alone."""
    t, d = 2000, 2048
    x = torch.ones(t, d, device="cuda", dtype=torch.bfloat16)
    bad = torch.arange(7, t, 13, device="cuda")
    x[bad, 100] = float("nan")
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    res = torch.zeros_like(x)
    y = torch.empty_like(x)
    B.mla_add_rmsnorm(x, res, res, B.MLA_OUT_BF16, w, 0.0, y, B.MLA_OUT_BF16)
    rows = torch.ones(t, dtype=torch.bool, device="cuda")
    rows[bad] = False
    assert torch.all(y[rows] == 1) and torch.all(y[~rows].isnan())


def test_norm_in_place_residual_and_stream():
    rng = np.random.default_rng(3)
    x, w, res = bf16(rng, (64, 1024)), bf16(rng, (1024,)), bf16(rng, (64, 1024))
    keep = res.clone()
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.mla_add_rmsnorm(x, res, res, B.MLA_OUT_BF16, w, 1e-6, y, B.MLA_OUT_BF16, stream=s)
    s.synchronize()
    assert torch.equal(res, (x.float() + keep.float()).to(torch.bfloat16))
    want, _ = L.rmsnorm(f64(x), f64(w), 1e-6, f64(keep))
    assert np.all(np.abs(f64(y) - want) <= np.abs(want) * (BF16_HALF + 2.0 ** -17))


def test_norm_special_values():
    """A zero row gives zeros; a NaN or an infinity spoils its own row only."""
    d = 384
    x = torch.ones(4, d, device="cuda", dtype=torch.bfloat16)
    x[1] = 0
    x[2, 200] = float("nan")
    x[3, 5] = float("inf")
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    _, y, _, sc = outputs(4, d, B.MLA_OUT_E4M3)
    B.mla_add_rmsnorm(x, None, None, 0, w, 0.0, y, B.MLA_OUT_E4M3, sc)
    v, s = y.float(), sc
    assert torch.all(v[0] == 448) and torch.allclose(s[:, 0] * 448, torch.ones(3, device="cuda"), atol=0, rtol=1e-6)
    assert torch.all(v[1].isnan())  # 0 * rsqrt(0): eps = 0 gives 0 * inf, as the formula
    B.mla_add_rmsnorm(x, None, None, 0, w, 1e-6, y, B.MLA_OUT_E4M3, sc)
    v = y.float()
    floor = np.float32(np.float32(1e-10) / np.float32(448))
    assert torch.all(v[1] == 0) and torch.all(sc[:, 1] == float(floor))
    assert torch.all(v[2].isnan()) and torch.all(sc[:, 2].isnan())
    # inf / inf is NaN in its block, finite / inf is 0 elsewhere
    assert sc[0, 3].isnan() and torch.all(sc[1:, 3] == float(floor)) and torch.all(v[3, 128:] == 0)


@pytest.mark.parametrize("t,d,pad", [(1, 1, 0), (1, 128, 0), (3, 130, 0), (17, 1001, 5), (64, 2048, 0), (300, 520, 8),
                                     (9, 127, 1), (2, 40000, 0)])
def test_quantize(t, d, pad):
    rng = np.random.default_rng(t + d)
    x = (bf16(rng, (t, d + pad)) * torch.from_numpy(10.0 ** rng.integers(-6, 6, (t, 1))).float().cuda()).to(torch.bfloat16)[:, :d]
    x[0, : min(d, 128)] = 0
    yw, y, scw, sc = outputs(t, d, B.MLA_OUT_E4M3, d + pad)
    B.mla_act_quantize(x, B.MLA_ACT_NONE, y, B.MLA_OUT_E4M3, sc)
    code, scale = L.quantize_f32(x.float().cpu().numpy())
    assert np.array_equal(sc.cpu().numpy(), scale)
    assert np.array_equal(f64(y), code)
    assert torch.all(yw[:, d:].float() == 7) and torch.all(scw[:, t:] == -5)


def test_quantize_special_values():
    x = torch.ones(4, 256, device="cuda", dtype=torch.bfloat16)
    x[1, 130] = float("nan")
    x[2, 3] = float("-inf")
    x[3] = torch.finfo(torch.bfloat16).min
    _, y, _, sc = outputs(4, 256, B.MLA_OUT_E4M3)
    B.mla_act_quantize(x, B.MLA_ACT_NONE, y, B.MLA_OUT_E4M3, sc)
    v = y.float()
    assert torch.all(v[0] == 448)
    assert torch.all(v[1, :128] == 448) and torch.all(v[1, 128:].isnan()) and sc[1, 1].isnan() and not sc[0, 1].isnan()
    assert sc[0, 2].isinf() and v[2, 3].isnan() and torch.all(v[2, 4:128] == 0) and torch.all(v[2, 128:] == 448)
    assert torch.all(v[3] == -448)


@pytest.mark.parametrize("y_dtype", [B.MLA_OUT_BF16, B.MLA_OUT_E4M3])
@pytest.mark.parametrize("t,d,pad", [(1, 1, 0), (4, 64, 0), (31, 2048, 0), (5, 333, 0), (130, 1024, 16)])
def test_silu_mul(t, d, pad, y_dtype):
    rng = np.random.default_rng(t * 31 + d)
    x = bf16(rng, (t, 2 * d + pad), 4.0)[:, :2 * d]
    x[0, 0], x[-1, d - 1] = -90.0, 90.0
    yw, y, _, sc = outputs(t, d, y_dtype, d + pad)
    B.mla_act_quantize(x, B.MLA_ACT_SILU_MUL, y, y_dtype, sc if y_dtype == B.MLA_OUT_E4M3 else None)
    want = L.silu_mul(f64(x))
    if y_dtype == B.MLA_OUT_BF16:
        assert np.all(np.abs(f64(y) - want) <= np.abs(want) * (BF16_HALF + 2.0 ** -14) + 2.0 ** -126)
    else:
        check_codes(y, sc, want, 2.0 ** -15)
    assert torch.all(yw[:, d:].float() == 7)


def test_silu_mul_of_infinities():
    inf, nan, big = float("inf"), float("nan"), 2.0 ** 127
    gate = [inf, inf, -inf, nan, big, -big, 0.0, -0.0, -80.0]
    up = [2.0, -2.0, 1.0, 1.0, 1.0, 1.0, inf, 3.0, 1.0]
    x = torch.tensor([gate + up], dtype=torch.bfloat16, device="cuda")
    y = torch.empty(1, len(gate), dtype=torch.bfloat16, device="cuda")
    B.mla_act_quantize(x, B.MLA_ACT_SILU_MUL, y, B.MLA_OUT_BF16, None)
    got = y[0].float().tolist()
    # g / (1 + e^-g): the gate itself, -inf / inf, and 0 times an infinity
    assert got[:2] == [inf, -inf] and all(np.isnan(got[i]) for i in (2, 3, 6))
    assert got[4] == big and got[5] == 0 and got[7] == 0
    assert abs(got[8] + 80 * np.exp(-80.0)) <= (BF16_HALF + 2.0 ** -14) * 80 * np.exp(-80.0)


# ------------------------------------------------------------------ products


def operands(rng, t, n, k, experts=1, integers=False, pad=0):
    """(a, sa, w, sw) as torch tensors; a in wider rows when pad > 0."""
    g = L.blocks(k)
    if integers:
        a = rng.integers(-2, 3, (t, k + pad)).astype(np.float32)
        w = rng.integers(-2, 3, (experts, n, k)).astype(np.float32)
        sa = 2.0 ** rng.integers(-1, 2, (g, t))
        sw = 2.0 ** rng.integers(-1, 2, (experts, L.blocks(n), g))
    else:
        a = rng.standard_normal((t, k + pad)).astype(np.float32) * 100
        w = rng.standard_normal((experts, n, k)).astype(np.float32) * 100
        sa = rng.uniform(0.001, 0.1, (g, t))
        sw = rng.uniform(0.0001, 0.01, (experts, L.blocks(n), g))
    dev = lambda v, kind: torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda().to(kind)  # noqa: E731
    return (dev(a, torch.float8_e4m3fn)[:, :k], dev(sa, torch.float32), dev(w, torch.float8_e4m3fn), dev(sw, torch.float32))


def check_product(out, want, mag, k, integers):
    live = ~np.isnan(want)
    got, want, mag = f64(out)[live], want[live], mag[live]
    half = BF16_HALF if out.dtype == torch.bfloat16 else F32_HALF
    if integers:
        assert np.array_equal(got, torch.from_numpy(want).to(out.dtype).double().numpy())
        return
    steps = (k / 32 + L.blocks(k) + 4) * 2.0 ** -19
    assert np.all(np.abs(got - want) <= half * np.abs(want) + steps * mag)


def run_gemm(rng, t, n, k, kind, integers, pad=0, out_pad=0):
    a, sa, w, sw = operands(rng, t, n, k, integers=integers, pad=pad)
    wide = torch.full((t, n + out_pad), 7.0, device="cuda", dtype=kind)
    out = wide[:, :n]
    B.mla_gemm_fp8(a, sa, w[0], sw[0], out, B.MLA_OUT_BF16 if kind == torch.bfloat16 else B.MLA_OUT_FP32)
    want, mag = L.gemm(f64(a), f64(sa), f64(w[0]), f64(sw[0]))
    assert B.mla_decode_device_error() == 0
    check_product(out, want, mag, k, integers)
    assert torch.all(wide[:, n:] == 7)


SIZES = [(1, 1, 16), (1, 576, 4096), (2, 128, 128), (7, 129, 144), (16, 127, 272), (17, 256, 384), (33, 1000, 2000),
         (64, 512, 1040), (65, 300, 128), (100, 1024, 1152), (128, 128, 2048), (129, 640, 512), (256, 260, 1024),
         (333, 1000, 2000), (513, 777, 272), (1030, 1300, 400)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", SIZES)
def test_gemm_exact_integers(t, n, k, kind):
    run_gemm(np.random.default_rng(t + n + k), t, n, k, kind, True, pad=16 * (t % 3), out_pad=n % 5)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", SIZES)
def test_gemm(t, n, k, kind):
    run_gemm(np.random.default_rng(t * n + k), t, n, k, kind, False)


LARGE = [(64, 4096, 4096), (100, 4100, 1040), (128, 8192, 2064), (200, 3000, 4096), (256, 8192, 1024), (300, 8200, 512),
         (512, 4096, 1000 // 16 * 16), (777, 2500, 1024), (1025, 4097, 400), (2000, 2300, 1168)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,n,k", LARGE)
def test_gemm_exact_integers_large(t, n, k, kind):
    """Sizes at which every form of the kernel is the one chosen (whole and split
    tiles of each width, pairs of CTAs), cut on all sides."""
    a, sa, w, sw = operands(np.random.default_rng(t * 3 + n + k), t, n, k, integers=True)
    for out_pad in (0, 3):
        wide = torch.full((t, n + out_pad), 7.0, device="cuda", dtype=kind)
        out = wide[:, :n]
        B.mla_gemm_fp8(a, sa, w[0], sw[0], out, B.MLA_OUT_BF16 if kind == torch.bfloat16 else B.MLA_OUT_FP32)
        assert B.mla_decode_device_error() == 0
        ad = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :k]
        wd = w[0].double() * sw[0].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        assert torch.equal(out, (ad @ wd.t()).to(kind)) and torch.all(wide[:, n:] == 7)


@pytest.mark.parametrize("counts,n,k", [([600, 0, 5, 411, 900, 33], 2100, 528), ([30] * 48, 1024, 1024),
                                        ([0, 2000, 1, 0], 1290, 1040), ([7] * 64, 4096, 512)])
def test_grouped_gemm_exact_integers_large(counts, n, k):
    t = sum(counts)
    a, sa, w, sw = operands(np.random.default_rng(t + n), t, n, k, len(counts), True)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    out = torch.full((t, n), 7.0, device="cuda")
    B.mla_grouped_gemm_fp8(a, sa, w, sw, torch.from_numpy(off).cuda(), out, B.MLA_OUT_FP32)
    assert B.mla_decode_device_error() == 0
    ad = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :k]
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        wd = w[e].double() * sw[e].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
        assert torch.equal(out[lo:hi], (ad[lo:hi] @ wd.t()).float())


@pytest.mark.parametrize("kind,unit", [(torch.bfloat16, 8), (torch.float32, 4)])
@pytest.mark.parametrize("n", [4095, 4097, 4100, 4104, 4160])
@pytest.mark.parametrize("t", [300, 4097])
def test_gemm_results_inside_wider_rows(t, n, kind, unit):
    """Tiles cut at the right edge and below, in rows of 16-byte multiples: what
    lies beside and below the results stays."""
    k = 256
    a, sa, w, sw = operands(np.random.default_rng(t + n), t, n, k, integers=True)
    ad = a.double() * sa.double().t().repeat_interleave(128, 1)
    wd = w[0].double() * sw[0].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    want = (ad @ wd.t()).to(kind)
    for width in (-(-n // unit) * unit, -(-n // unit) * unit + unit):
        wide = torch.full((t + 3, width), 7.0, device="cuda", dtype=kind)
        B.mla_gemm_fp8(a, sa, w[0], sw[0], wide[:t, :n], B.MLA_OUT_BF16 if kind == torch.bfloat16 else B.MLA_OUT_FP32)
        assert B.mla_decode_device_error() == 0
        assert torch.equal(wide[:t, :n], want)
        assert torch.all(wide[t:] == 7) and torch.all(wide[:, n:] == 7)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,n", [([3000, 37, 0, 2100], 4104), ([130, 0, 129, 1, 300], 1096)])
def test_grouped_gemm_large_unowned_rows(counts, n, kind):
    k, head, tail = 256, 5, 70
    t = head + sum(counts) + tail
    a, sa, w, sw = operands(np.random.default_rng(t + n), t, n, k, len(counts), True)
    off = (head + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    out = torch.full((t, n), 7.0, device="cuda", dtype=kind)
    B.mla_grouped_gemm_fp8(a, sa, w, sw, torch.from_numpy(off).cuda(), out,
                           B.MLA_OUT_BF16 if kind == torch.bfloat16 else B.MLA_OUT_FP32)
    assert B.mla_decode_device_error() == 0
    ad = a.double() * sa.double().t().repeat_interleave(128, 1)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        wd = w[e].double() * sw[e].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        assert torch.equal(out[lo:hi], (ad[lo:hi] @ wd.t()).to(kind))
    assert torch.all(out[:head] == 7) and torch.all(out[off[-1]:] == 7)


def run_grouped(rng, counts, n, k, kind, integers, head=0, tail=0):
    t = head + int(sum(counts)) + tail
    a, sa, w, sw = operands(rng, t, n, k, len(counts), integers)
    off = head + np.concatenate([[0], np.cumsum(counts)])
    out = torch.full((t, n), 7.0, device="cuda", dtype=kind)
    B.mla_grouped_gemm_fp8(a, sa, w, sw, torch.from_numpy(off.astype(np.int32)).cuda(), out,
                           B.MLA_OUT_BF16 if kind == torch.bfloat16 else B.MLA_OUT_FP32)
    want, mag = L.grouped_gemm(f64(a), f64(sa), f64(w), f64(sw), off)
    assert B.mla_decode_device_error() == 0
    check_product(out, want, mag, k, integers)
    assert torch.all(out[:head] == 7) and torch.all(out[t - tail:] == 7)  # rows that no expert owns


COUNTS = [([1], 128, 128), ([0, 3, 0, 17, 1], 130, 272), ([5, 0, 0, 200, 40, 16, 130], 328, 1040),
          ([0, 0, 700], 256, 512), (list(range(40)), 96, 144), ([300, 1, 299, 257], 520, 384)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("integers", [True, False])
@pytest.mark.parametrize("counts,n,k", COUNTS)
def test_grouped_gemm(counts, n, k, integers, kind):
    run_grouped(np.random.default_rng(sum(counts) + n + k), counts, n, k, kind, integers)


def test_grouped_gemm_unowned_rows():
    run_grouped(np.random.default_rng(5), [9, 0, 33], 200, 256, torch.bfloat16, True, head=5, tail=70)


def test_grouped_gemm_all_empty_and_many_experts():
    run_grouped(np.random.default_rng(6), [0, 0, 0], 64, 128, torch.bfloat16, True, tail=3)
    rng = np.random.default_rng(7)
    run_grouped(rng, rng.integers(0, 3, B.MLA_GEMM_MAX_EXPERTS), 16, 64, torch.float32, True)


@pytest.mark.parametrize("off", [[0, 5, -3, 10], [0, 4, 11, 10], [-2, 4, 6, 10], [0, 5, 2 ** 31 - 1, 10]])
def test_grouped_gemm_malformed_offsets(off):
    """A broken entry costs its experts their rows and sets the error word;
    nothing outside the arrays is touched (checked by the kernel before use)."""
    rng = np.random.default_rng(8)
    a, sa, w, sw = operands(rng, 10, 128, 128, 3, True)
    out = torch.full((10, 128), 7.0, device="cuda")
    B.mla_grouped_gemm_fp8(a, sa, w, sw, torch.tensor(off, dtype=torch.int32, device="cuda"), out, B.MLA_OUT_FP32)
    assert B.mla_decode_device_error() == 0x701
    owner = [-1] * 10
    for e in range(3):
        if 0 <= off[e] <= off[e + 1] <= 10:
            for m in range(off[e], off[e + 1]):
                owner[m] = e
    for m in range(10):
        if owner[m] < 0:
            assert torch.all(out[m] == 7)
        else:
            e = owner[m]
            want, _ = L.gemm(f64(a[m:m + 1]), f64(sa[:, m:m + 1]), f64(w[e]), f64(sw[e]))
            assert np.array_equal(f64(out[m:m + 1]), want)


def test_gemm_non_finite_operands_stay_in_their_row_and_column():
    rng = np.random.default_rng(9)
    for t, n in [(5, 200), (300, 400)]:
        a, sa, w, sw = operands(rng, t, n, 384, integers=True)
        a, w = a.clone(), w[0].clone()
        a.view(torch.uint8)[2, 150] = 0x7F  # NaN code
        w.view(torch.uint8)[131, 10] = 0xFF
        sa[1, 4] = float("inf")
        out = torch.empty(t, n, device="cuda")
        B.mla_gemm_fp8(a, sa, w, sw[0], out, B.MLA_OUT_FP32)
        bad = torch.zeros(t, n, dtype=torch.bool, device="cuda")
        bad[2], bad[:, 131] = True, True
        assert torch.all(out[bad].isnan())
        bad[4] = True  # infinity times the block's sums: +-inf, or NaN where the sum is 0
        assert not torch.any(out[4].isfinite()) and torch.all(out[~bad].isfinite())


def test_gemm_same_bits_every_call_and_graph():
    rng = np.random.default_rng(10)
    for t, n, k in [(3, 576, 2048), (200, 512, 1024), (600, 1024, 512)]:
        a, sa, w, sw = operands(rng, t, n, k)
        out = [torch.empty(t, n, device="cuda") for _ in range(3)]
        B.mla_gemm_fp8(a, sa, w[0], sw[0], out[0], B.MLA_OUT_FP32)
        B.mla_gemm_fp8(a, sa, w[0], sw[0], out[1], B.MLA_OUT_FP32)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            B.mla_gemm_fp8(a, sa, w[0], sw[0], out[2], B.MLA_OUT_FP32, stream=s)
        g.replay()
        torch.cuda.synchronize()
        bits = [o.view(torch.int32) for o in out]  # an operand beyond 448 is a NaN code: compare bits, not values
        assert torch.equal(bits[0], bits[1]) and torch.equal(bits[0], bits[2])


def test_rows_past_32_bit_offsets():
    """Output offsets past 2^31 elements and operand rows past 2^32 bytes."""
    t, n, k, ld = 70000, 40, 64, 65536
    a8 = torch.zeros(t, ld, dtype=torch.uint8, device="cuda")  # 4.6 GB, rows 64 KB apart
    rng = np.random.default_rng(11)
    a, sa, w, sw = operands(rng, t, n, k, integers=True)
    a8[:, :k] = a.view(torch.uint8)
    wide = torch.empty(t, ld, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 100:100 + n]
    B.mla_gemm_fp8(a8[:, :k], sa, w[0], sw[0], out, B.MLA_OUT_BF16)
    want, mag = L.gemm(f64(a[-300:]), f64(sa[:, -300:]), f64(w[0]), f64(sw[0]))
    check_product(out[-300:], want, mag, k, True)
    y, sc = a8[:, 128:128 + n], torch.empty(1, t, device="cuda")
    B.mla_act_quantize(out, B.MLA_ACT_NONE, y, B.MLA_OUT_E4M3, sc)
    code, scale = L.quantize_f32(out[-300:].float().cpu().numpy())
    assert np.array_equal(f64(y[-300:].view(torch.float8_e4m3fn)), code) and np.array_equal(sc[:, -300:].cpu().numpy(), scale)


def test_chain_norm_to_product():
    """The norm's e4m3 rows and scales feed the product as they are."""
    rng = np.random.default_rng(12)
    t, d, n = 50, 1024, 384
    x, wt = bf16(rng, (t, d)), bf16(rng, (d,))
    y, sc = torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(8, t, device="cuda")
    B.mla_add_rmsnorm(x, None, None, 0, wt, 1e-6, y, B.MLA_OUT_E4M3, sc)
    _, _, w, sw = operands(rng, 1, n, d)
    out = torch.empty(t, n, device="cuda")
    B.mla_gemm_fp8(y, sc, w[0], sw[0], out, B.MLA_OUT_FP32)
    want, mag = L.gemm(f64(y), f64(sc), f64(w[0]), f64(sw[0]))
    check_product(out, want, mag, d, False)
