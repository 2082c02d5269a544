"""The forms of the FP8 products, one by one, against the float64 definition.

Operands are small integers and scales powers of two, so every sum is exact in
fp32 and the result has to equal the rounded exact value, bit for bit."""

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
