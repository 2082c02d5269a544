"""The forms of the FP8 products, one by one, against the float64 definition.

The products choose their form by an estimate of the time, so the sizes of a test
do not say which one it reaches; these ask for each.  Where operands are small
integers and scales powers of two, every sum is exact in fp32 and the result has
to equal the rounded exact value, bit for bit.  Other operands: a product rounds
once per 32-wide step (its 33 summands aligned to the largest with at least 25 bits
kept, 33 * 2^-25 < 2^-19), twice per block of 128 and once per part of k, below
(k / 32 + blocks + parts + 4) * 2^-19 of the sum of the terms' magnitudes; then half
a step of the output type."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_layer_ref as L
from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    B.mla_decode_device_error(reset=True)
    yield
    assert B.mla_decode_device_error(reset=True) == 0


def operands(rng, t, n, k, experts=1):
    """(a, sa, w, sw): codes -2 .. 2, scales 1/2, 1, 2."""
    g = L.blocks(k)
    dev = lambda v, kind: torch.from_numpy(v.astype(np.float32)).cuda().to(kind)  # noqa: E731
    return (dev(rng.integers(-2, 3, (t, k)), torch.float8_e4m3fn), dev(2.0 ** rng.integers(-1, 2, (g, t)), torch.float32),
            dev(rng.integers(-2, 3, (experts, n, k)), torch.float8_e4m3fn),
            dev(2.0 ** rng.integers(-1, 2, (experts, L.blocks(n), g)), torch.float32))


def exact(a, sa, w, sw):
    """The product of one expert in float64 (exact here)."""
    n, k = w.shape
    a = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :k]
    w = w.double() * sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return a @ w.t()


def in_form(a, sa, w, sw, off, out, tile, parts, give_up=-1):
    """mla_gemm_fp8_in_form on contiguous operands and an `out` with contiguous columns."""
    rc = B.load().mla_gemm_fp8_in_form(
        a.data_ptr(), a.stride(0), sa.data_ptr(), sa.stride(0), w.data_ptr(), w.stride(-2), sw.data_ptr(),
        None if off is None else off.data_ptr(), w.shape[0], a.shape[0], w.shape[1], a.shape[1], out.data_ptr(),
        B.MLA_OUT_BF16 if out.dtype == torch.bfloat16 else B.MLA_OUT_FP32, out.stride(0), tile, parts, give_up,
        torch.cuda.current_stream().cuda_stream)
    assert rc == B.MLA_OK, B.load().mla_decode_last_error_string()


FORMS = [(16, 1), (16, 2), (16, 4), (16, 8), (32, 1), (32, 2), (32, 4), (32, 8), (64, 1), (64, 2), (64, 4), (64, 8),
         (128, 1), (256, 1)]

KINDS = [torch.bfloat16, torch.float32]
# one row and column; both cut inside a tile and a short last block of k; several
# tiles each way, cut; whole tiles; rows of results that are not 16 bytes apart
DENSE = [(1, 1, 2048, 0), (37, 200, 2064, 0), (300, 391, 2192, 5), (512, 768, 2048, 0), (261, 1000, 2304, 8)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,n,k,pad", DENSE)
@pytest.mark.parametrize("tile,parts", FORMS)
def test_dense(tile, parts, t, n, k, pad, kind):
    a, sa, w, sw = operands(np.random.default_rng(t + n + k), t, n, k)
    wide = torch.full((t + 2, n + pad), 7.0, device="cuda", dtype=kind)
    in_form(a, sa, w, sw, None, wide[:t, :n], tile, parts)
    assert torch.equal(wide[:t, :n], exact(a, sa, w[0], sw[0]).to(kind))
    assert torch.all(wide[t:] == 7) and torch.all(wide[:, n:] == 7)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,n,k,pad", [([0, 3, 0, 17, 1], 130, 2064, 0), ([300, 1, 0, 257, 64], 264, 2048, 8),
                                            ([0, 0, 0], 64, 2048, 0), ([1, 0, 2, 5] * 20, 96, 2176, 3)])
@pytest.mark.parametrize("tile,parts", FORMS)
def test_grouped(tile, parts, counts, n, k, pad, kind):
    """Experts without rows, rows without an expert before and after, clusters
    and CTAs without a tile."""
    head, tail = 5, 70
    off = (head + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    t = int(off[-1]) + tail
    a, sa, w, sw = operands(np.random.default_rng(t + n), t, n, k, len(counts))
    wide = torch.full((t, n + pad), 7.0, device="cuda", dtype=kind)
    in_form(a, sa, w, sw, torch.from_numpy(off).cuda(), wide[:, :n], tile, parts)
    want = torch.full((t, n), 7.0, device="cuda", dtype=kind)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        want[lo:hi] = exact(a[lo:hi], sa[:, lo:hi], w[e], sw[e]).to(kind)
    assert torch.equal(wide[:, :n], want) and torch.all(wide[:, n:] == 7)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tile,parts", FORMS)
def test_other_operands(tile, parts, kind):
    """Operands over the whole range of the codes, scales of many magnitudes."""
    t, n, k = 150, 300, 4096
    rng = np.random.default_rng(tile * parts)
    dev = lambda v, to: torch.from_numpy(v.astype(np.float32)).cuda().to(to)  # noqa: E731
    a = dev(np.clip(rng.standard_normal((t, k)) * 100, -448, 448), torch.float8_e4m3fn)
    w = dev(np.clip(rng.standard_normal((1, n, k)) * 100, -448, 448), torch.float8_e4m3fn)
    sa = dev(10.0 ** rng.uniform(-6, 2, (L.blocks(k), t)), torch.float32)
    sw = dev(10.0 ** rng.uniform(-6, 2, (1, L.blocks(n), L.blocks(k))), torch.float32)
    out = torch.empty(t, n, device="cuda", dtype=kind)
    in_form(a, sa, w, sw, None, out, tile, parts)
    f64 = lambda v: v.double().cpu().numpy()  # noqa: E731
    want, mag = L.gemm(f64(a), f64(sa), f64(w[0]), f64(sw[0]))
    half = 2.0 ** -8 if kind == torch.bfloat16 else 2.0 ** -24
    steps = (k / 32 + L.blocks(k) + parts + 4) * 2.0 ** -19
    assert np.all(np.abs(f64(out) - want) <= half * np.abs(want) + steps * mag)


@pytest.mark.parametrize("tile,parts", FORMS)
def test_non_finite(tile, parts):
    """NaN codes and infinite or NaN scales reach the results that use them and
    no other, whether an expert's rows, the next one's or nobody's lie beside."""
    counts, n, k = [70, 0, 61, 130], 260, 2304
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    t = int(off[-1]) + 9
    a, sa, w, sw = operands(np.random.default_rng(tile + parts), t, n, k, len(counts))
    a[0], a[69], a[140], w[0, 131], w[3, 259] = 1, 1, 1, 1, 1  # no block of these sums to 0 by chance
    sa[2, 0], sa[17, 69] = float("inf"), float("nan")
    a.view(torch.uint8)[140, 2303] = 0x7F
    w.view(torch.uint8)[0, 131, 5] = 0xFF
    sw[3, 2, 9] = float("nan")
    a.view(torch.uint8)[off[-1]:] = 0x7F  # rows without an expert
    sa[:, off[-1]:] = float("nan")
    out = torch.full((t, n), 7.0, device="cuda")
    in_form(a, sa, w, sw, torch.from_numpy(off).cuda(), out, tile, parts)
    want = torch.full((t, n), 7.0, device="cuda", dtype=torch.float64)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        for b in range(L.blocks(k)):
            cols = slice(128 * b, min(k, 128 * b + 128))
            if b == 0:
                want[lo:hi] = 0
            term = a[lo:hi, cols].double() @ w[e][:, cols].double().t()
            want[lo:hi] += term * sa[b, lo:hi, None].double() * sw[e, :, b].repeat_interleave(128)[:n].double()
    assert torch.all(want[69].isnan()) and torch.all(want[140].isnan()) and torch.all(want[:70, 131].isnan())
    assert torch.all(want[131:261, 256:].isnan()) and int(want.isfinite().sum()) > 200 * n // 2
    want = want.float()
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(0.0, 1e38, -1e38), want.nan_to_num(0.0, 1e38, -1e38))


@pytest.mark.parametrize("tile,parts", FORMS)
def test_same_bits_every_call(tile, parts):
    t, n, k = 200, 520, 4096
    rng = np.random.default_rng(3)
    dev = lambda v, to: torch.from_numpy(v.astype(np.float32)).cuda().to(to)  # noqa: E731
    a = dev(np.clip(rng.standard_normal((t, k)) * 100, -448, 448), torch.float8_e4m3fn)
    w = dev(np.clip(rng.standard_normal((1, n, k)) * 100, -448, 448), torch.float8_e4m3fn)
    sa, sw = dev(rng.uniform(0.1, 1, (L.blocks(k), t)), torch.float32), dev(rng.uniform(0.1, 1, (1, 5, L.blocks(k))), torch.float32)
    outs = [torch.empty(t, n, device="cuda") for _ in range(4)]
    for out in outs:
        in_form(a, sa, w, sw, None, out, tile, parts)
    assert all(torch.equal(outs[0], out) for out in outs[1:])


def test_the_call_takes_the_form_it_names():
    """A product's bits are those of the form that mla_gemm_fp8_form names for it
    on this device (forms add up in different orders), and the forms named over
    the sizes are all among those tested here."""
    rng = np.random.default_rng(4)
    lib, seen = B.load(), set()
    named = [ctypes.c_int() for _ in range(3)]
    for t, n, k in [(1, 576, 4096), (20, 1000, 8192), (64, 4096, 16384), (64, 7168, 16384), (100, 4096, 4096),
                    (500, 2048, 4096), (1500, 4096, 2048), (64, 36864, 7168)]:
        a = torch.from_numpy(rng.integers(1, 0x7E, (t, k)).astype(np.uint8)).cuda()
        w = torch.from_numpy(rng.integers(1, 0x7E, (1, 1024, k)).astype(np.uint8)).cuda().repeat(1, -(-n // 1024), 1)[:, :n]
        w = w.contiguous()
        sa = torch.from_numpy(rng.uniform(0.5, 2, (L.blocks(k), t)).astype(np.float32)).cuda()
        sw = torch.from_numpy(rng.uniform(0.5, 2, (1, L.blocks(n), L.blocks(k))).astype(np.float32)).cuda()
        out, again = torch.empty(t, n, device="cuda"), torch.empty(t, n, device="cuda")
        assert lib.mla_gemm_fp8_form(t, n, k, 1, 0, B.MLA_OUT_FP32, out.data_ptr(), n, 0, None,
                                     *[ctypes.byref(v) for v in named]) == B.MLA_OK
        form = (named[0].value, named[1].value)
        assert form in FORMS
        seen.add(form)
        B.mla_gemm_fp8(a, sa, w[0], sw[0], out, B.MLA_OUT_FP32)
        in_form(a, sa, w, sw, None, again, *form)
        assert torch.equal(out, again)
    assert len(seen) >= 5


def owned(off, t):
    """Rows of each expert: its range, unless that is no range within [0, t] or
    begins before the end of an earlier one."""
    rows, end = [], 0
    for lo, hi in zip(off[:-1], off[1:]):
        ok = 0 <= lo <= hi <= t
        rows.append(range(lo, hi) if ok and (lo >= end or lo == hi) else range(0))
        if ok and hi > lo:
            end = max(end, hi)
    return rows


def broken_offsets():
    rng = np.random.default_rng(0)
    many = np.sort(rng.integers(0, 201, 71))  # three groups of 32 experts
    for i, v in [(5, -1), (30, 201), (31, 0), (33, 200), (50, 3), (64, 0)]:
        many[i] = v
    return [([0, 40, 0, 40], 40), ([0, 40, 0, 40, 0, 40, 0, 40], 40), ([0, 30, 20, 40], 40), ([10, 5, 20, 12, 25, 40], 40),
            ([3, 3, 50, 40, 50, 60, 20, 64], 64), ([0] * 33 + [9, 4, 30], 30), (many.tolist(), 200)]


@pytest.mark.parametrize("tile,parts", FORMS)
@pytest.mark.parametrize("off,t", broken_offsets())
def test_no_row_has_two_owners(off, t, tile, parts):
    """Offsets that descend: overlapping ranges are refused on the device, and
    the rows that are owned are right in every form."""
    n, k, experts = 136, 2048, len(off) - 1
    a, sa, w, sw = operands(np.random.default_rng(t + experts), t, n, k, experts)
    out = torch.full((t, n), 7.0, device="cuda")
    in_form(a, sa, w, sw, torch.tensor(off, dtype=torch.int32, device="cuda"), out, tile, parts)
    assert B.mla_decode_device_error(reset=True) == 0x701
    want = torch.full_like(out, 7.0)
    for e, rows in enumerate(owned(off, t)):
        if len(rows):
            r = slice(rows.start, rows.stop)
            want[r] = exact(a[r], sa[:, r], w[e], sw[e]).float()
    assert torch.equal(out, want)


@pytest.mark.parametrize("tile,parts", FORMS)
def test_offsets_from_the_kernel_before(tile, parts):
    """The offsets are results of a long kernel that is still running when the
    product's CTAs become resident (a norm's residual output, whose last row they
    are: 0 + bits, exact), call by call and replayed from a graph."""
    experts, t, n, k, rows = 64, 192, 136, 2048, 20000
    rng = np.random.default_rng(tile + parts)
    a, sa, w, sw = operands(rng, t, n, k, experts)
    x = torch.zeros(rows, experts + 1, dtype=torch.bfloat16, device="cuda")
    weight, y = torch.ones(experts + 1, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    source = torch.zeros(rows, experts + 1, device="cuda")
    copied = torch.zeros_like(source)
    off = copied[-1].view(torch.int32)
    out = torch.empty(t, n, device="cuda")

    def step():
        B.mla_add_rmsnorm(x, source, copied, B.MLA_OUT_FP32, weight, 1.0, y, B.MLA_OUT_BF16)
        in_form(a, sa, w, sw, off, out, tile, parts)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        now = np.sort(np.concatenate([[0, t], rng.integers(0, t + 1, experts - 1)])).astype(np.int32)
        source[-1].view(torch.int32).copy_(torch.from_numpy(now))
        torch.cuda.synchronize()
        graph.replay() if i % 2 else step()
        want = torch.cat([exact(a[lo:hi], sa[:, lo:hi], w[e], sw[e]) for e, (lo, hi) in enumerate(zip(now[:-1], now[1:]))])
        assert torch.equal(out, want.float())


@pytest.mark.parametrize("tile,parts,k,warp", [(16, 8, 2048, 0), (16, 8, 2048, 3), (16, 2, 4096, 1), (32, 4, 1024, 5),
                                               (64, 8, 4096, 7), (64, 2, 512, 4), (16, 1, 1024, 2), (64, 1, 2048, 6)])
def test_a_warp_that_gives_up_ends_the_kernel(tile, parts, k, warp):
    """One epilogue warp of one CTA gives up while all others go on: the kernel
    ends, says so, and the next call is right."""
    t, n = min(tile, 40), 300
    a, sa, w, sw = operands(np.random.default_rng(k + warp), t, n, k)
    out = torch.empty(t, n, device="cuda")
    in_form(a, sa, w, sw, None, out, tile, parts, warp)
    assert B.mla_decode_device_error(reset=True) == 0x718
    in_form(a, sa, w, sw, None, out, tile, parts)
    assert B.mla_decode_device_error() == 0
    assert torch.equal(out, exact(a, sa, w[0], sw[0]).float())
