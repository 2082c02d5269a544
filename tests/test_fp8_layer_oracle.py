"""Pins of the FP8 layer oracle (CPU): the e4m3 rounding against torch's cast,
the quantiser against its definition, the products against element loops."""

import numpy as np
import torch

from oracle import fp8_layer_ref as L


def test_round_e4m3_matches_the_format():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000),
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 448.0, -448.0, np.nan]])
    v = np.clip(v, -448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    got = L.round_e4m3(v)
    assert np.array_equal(got, want, equal_nan=True) and np.array_equal(np.signbit(got[:-1]), np.signbit(want[:-1]))
    assert L.round_e4m3(np.array([1e9, -1e9])).tolist() == [448.0, -448.0]


def test_quantizer_hits_the_maximum_and_half_a_step():
    rng = np.random.default_rng(1)
    v = (rng.standard_normal((5, 300)) * 10.0 ** rng.integers(-4, 4, (5, 1))).astype(np.float32)
    code, scale = L.quantize_f32(v)
    assert scale.shape == (3, 5) and np.abs(code).max() == 448
    deq = code * L.spread(scale.astype(np.float64), 300)
    s = L.spread(scale.astype(np.float64), 300)
    assert np.all(np.abs(deq - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) * (1 + 2.0 ** -20))
    zero, zs = L.quantize_f32(np.zeros((1, 4), np.float32))
    assert np.all(zero == 0) and zs[0, 0] == np.float32(np.float32(1e-10) / np.float32(448))


def test_norm_and_gate_by_hand():
    y, h = L.rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0, [[0.0, 0.0]])
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]) and np.array_equal(h, [[3.0, 4.0]])
    assert np.allclose(L.silu_mul([[0.0, 1.0, 5.0, 2.0]]), [[0.0, 2.0 / (1 + np.exp(-1.0))]])


def test_products_against_loops():
    rng = np.random.default_rng(2)
    a, w = rng.integers(-3, 4, (4, 272)), rng.integers(-3, 4, (2, 130, 272))
    sa, sw = rng.uniform(0.5, 2, (3, 4)), rng.uniform(0.5, 2, (2, 2, 3))
    out, mag = L.grouped_gemm(a, sa, w, sw, [1, 1, 3])
    assert np.isnan(out[[0, 3]]).all()
    for m in (1, 2):
        for n in (0, 127, 128, 129):
            terms = [a[m, k] * w[1, n, k] * sa[k // 128, m] * sw[1, n // 128, k // 128] for k in range(272)]
            assert abs(out[m, n] - sum(terms)) < 1e-9 and abs(mag[m, n] - sum(map(abs, terms))) < 1e-9
