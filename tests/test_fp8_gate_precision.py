"""The gated unit's fp32 value, closely.

A bf16 or e4m3 result hides it; the scale of a block that holds one element that
is not zero is that element's magnitude over 448, in fp32.

Bound, from the steps of g / (1 + e^-g) with e = expf(-|g|): expf is within 2 ulp
(2^-22 relative), 1 + e rounds once (2^-24) and carries e's error times e / (1 + e),
g * e rounds once (2^-24), the corrected quotient is within an ulp (2^-23).  A
positive gate collects 2^-23 + 2^-24 + 2^-23, a negative one, whose numerator holds
e too, 2^-22 / (1 + e) + 2^-24 + 2^-24 + 2^-23: both below 2^-21.  The product with
a power of two is exact, the scale rounds once (2^-24)."""

import numpy as np
import pytest
import torch

from oracle import fp8_layer_ref as L
from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu

VALUE = 2.0 ** -21


@pytest.fixture(autouse=True)
def no_device_error():
    B.mla_decode_device_error(reset=True)
    yield
    assert B.mla_decode_device_error(reset=True) == 0


@pytest.mark.parametrize("power", [60, 100])
@pytest.mark.parametrize("at", [0, 77])
@pytest.mark.parametrize("dim", [128, 120, 117])
def test_value_of_every_gate(dim, at, power):
    """Every bf16 gate between 2^-12 and 87 in magnitude, both signs; rows read by
    16-byte pieces and element by element."""
    bits = torch.arange(0x3980, 0x42AE, dtype=torch.int32).to(torch.int16)  # 2^-12 .. 86.5
    gates = bits.view(torch.bfloat16)
    gates = torch.cat([gates, -gates])
    x = torch.zeros(gates.numel(), 2 * dim, dtype=torch.bfloat16)
    x[:, at], x[:, dim + at] = gates, 2.0 ** power
    y = torch.empty(gates.numel(), dim, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(1, gates.numel(), device="cuda")
    B.mla_act_quantize(x.cuda(), B.MLA_ACT_SILU_MUL, y, B.MLA_OUT_E4M3, scale)
    g = gates.double().numpy()
    want = np.abs(g / (1.0 + np.exp(-g))) * 2.0 ** power
    want = np.maximum(want, 1e-10)  # the floor of a block's maximum: gates below -70 with 2^60
    got = scale[0].double().cpu().numpy() * 448
    assert np.all(np.abs(got - want) <= (VALUE + 2.0 ** -24) * want)


def test_codes_on_the_other_side_of_a_border():
    """Codes differ from those of the exact value, at the same scales, only where
    it lies within its error of a border between two codes.  The fp32 value, the
    reciprocal of the scale and their product are off by VALUE + 3 * 2^-24 together;
    borders are at least 1/16 of a value apart, so at most a share of 2 * 16 times
    that of the codes may differ, and five standard deviations of their number."""
    t, d = 4096, 2048
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((t, 2 * d)).astype(np.float32) * 2).to(torch.bfloat16)
    y = torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(L.blocks(d), t, device="cuda")
    B.mla_act_quantize(x.cuda(), B.MLA_ACT_SILU_MUL, y, B.MLA_OUT_E4M3, scale)
    want = L.silu_mul(x.double().numpy())
    codes = L.round_e4m3(want / L.spread(scale.double().cpu().numpy(), d))
    got = y.double().cpu().numpy()
    differ = got != codes
    assert np.all(np.abs(got - codes) <= np.maximum(np.abs(codes) / 8, 2.0 ** -9))  # the neighbour, at most
    expected = 2 * 16 * (VALUE + 3 * 2.0 ** -24) * t * d
    assert int(differ.sum()) <= expected + 5 * np.sqrt(expected)
