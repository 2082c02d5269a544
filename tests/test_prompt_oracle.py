"""The float64 oracle of the prompt's operators against what the definitions imply."""

import numpy as np
import pytest

from oracle import prompt_ref as O

RNG = np.random.default_rng(0)


def test_rotation_depends_on_the_distance_alone():
    f = O.rope_frequencies(64, 1e4)
    t = O.rope_table(0, 300, f)
    for neox in (False, True):
        q, k = RNG.standard_normal((2, 64))
        dots = [O.rope(q, t[i + 37], neox) @ O.rope(k, t[i], neox) for i in (0, 5, 200)]
        assert np.allclose(dots, dots[0], atol=1e-12)
        assert np.allclose(O.rope(q, t[0], neox), q)


def test_layouts_are_permutations_of_each_other():
    t = O.rope_table(9, 1, O.rope_frequencies(8, 100.0))[0]
    x = RNG.standard_normal(8)
    order = np.r_[0:8:2, 1:8:2]
    assert np.allclose(O.rope(x, t, False)[order], O.rope(x[order], t, True))


def test_scaled_frequencies():
    f = O.rope_frequencies(64, 1e4)
    assert np.allclose(O.rope_frequencies(64, 1e4, "linear", 8.0), f / 8)
    y = O.rope_frequencies(64, 1e4, "yarn", 40.0, 4096)
    assert np.all(y <= f) and np.all(y >= f / 40 * (1 - 1e-12))
    turns = 4096 * f / (2 * np.pi)
    assert np.allclose(y[turns > 40], f[turns > 40]) and np.allclose(y[turns < 0.7], f[turns < 0.7] / 40)
    assert np.all(np.diff(y) < 0)


def test_merge_of_parts_is_the_whole():
    q, k, v = RNG.standard_normal((7, 2, 192)), RNG.standard_normal((50, 2, 192)), RNG.standard_normal((50, 2, 128))
    whole = O.prefill(q, k, v, [0, 7], [0, 50], 0.07, False)
    a = O.prefill(q, k[:13], v[:13], [0, 7], [0, 13], 0.07, False)
    b = O.prefill(q, k[13:], v[13:], [0, 7], [0, 37], 0.07, False)
    out, lse = O.merge(a[0], a[1], b[0], b[1])
    assert np.allclose(out, whole[0]) and np.allclose(lse, whole[1])
    none = O.prefill(q, k[:0], v[:0], [0, 7], [0, 0], 0.07, False)
    out, lse = O.merge(*whole[:2], *none[:2])
    assert np.array_equal(out, whole[0]) and np.array_equal(lse, whole[1])
    assert not none[0].any() and np.all(np.isneginf(none[1]))


def test_causal_rows_are_the_last_ones():
    q, k, v = RNG.standard_normal((5, 1, 192)), RNG.standard_normal((9, 1, 192)), RNG.standard_normal((9, 1, 128))
    out, lse, _, _ = O.prefill(q, k, v, [0, 5], [0, 9], 0.1, True)
    for i in range(5):
        one = O.prefill(q[i:i + 1], k[:5 + i], v[:5 + i], [0, 1], [0, 5 + i], 0.1, False)
        assert np.allclose(out[i], one[0][0]) and np.allclose(lse[i], one[1][0])
    out, lse, _, _ = O.prefill(q, k[:2], v[:2], [0, 5], [0, 2], 0.1, True)
    assert not out[:3].any() and np.all(np.isneginf(lse[:3])) and np.allclose(out[3], v[0])


@pytest.mark.parametrize("page", [32, 64])
def test_gathered_slots(page):
    table = np.array([[4, 2, 9], [7, -1, -1]])
    slots = O.gather_rows(table, [page - 1, 3], [0, 3, 5], page, 6)
    assert slots.tolist() == [4 * page + page - 1, 2 * page, 2 * page + 1, 7 * page + 3, 7 * page + 4, -1]
