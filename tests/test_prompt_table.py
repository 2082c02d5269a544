"""Large rotary tables, whose threads have four rows each, against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from oracle import prompt_ref as O
from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu
SCALINGS = {"plain": B.MLA_ROPE_PLAIN, "linear": B.MLA_ROPE_LINEAR, "yarn": B.MLA_ROPE_YARN}


def table(first, n, dim, scaling, factor, magnitude=1.0):
    t = torch.full((n, dim), 9.0, device="cuda")
    B.mla_rope_table(t, first, 1e4, SCALINGS[scaling], factor, 4096, 32.0, 1.0, magnitude)
    return t


# 64 columns go by 16-byte pieces, 30 one by one; neither number of rows fills its last block
LARGE = [(0, 30001, 64, "yarn", 40.0, 1.0), (1000, 20011, 30, "linear", 8.0, 1.0), (500001, 25000, 40, "plain", 1.0, 0.7),
         ((1 << 31) - 30000, 30000, 64, "plain", 1.0, 1.0)]


@pytest.mark.parametrize("first,n,dim,scaling,factor,magnitude", LARGE)
def test_large_tables(first, n, dim, scaling, factor, magnitude):
    """In units of 2^-24, for an angle y of at most pi / 4 after the reduction.  The turn is
    cut to 2^-32 (0.04 as an angle); y has three roundings (to fp32, the constant's, the
    product's), 3 * pi / 4, of which the sine and the cosine take at most the share
    sqrt(1/2): 1.7.  The polynomials: terms left out below 2e-9 (0.04); z = y^2 rounded,
    at most 0.62 times the half that it weighs in the cosine (0.3); the last
    coefficient's sum, 0.5 times 0.62 (0.3); the final sum (0.5).  The product with the
    magnitude and the magnitude's own rounding: 2.  Together below 5, of the magnitude.
    Frequencies: two powers (2^-52 each) and five roundings of 2^-53 in the kernel's and the
    oracle's chains together, of the angle."""
    got = table(first, n, dim, scaling, factor, magnitude).double().cpu().numpy()
    want = O.rope_table(first, n, O.rope_frequencies(dim, 1e4, scaling, factor), magnitude)
    tol = (5 * 2.0 ** -24 + 5 * 2.0 ** -52 * (first + n)) * magnitude
    assert np.abs(got - want).max() <= tol


@pytest.mark.parametrize("dim", [64, 30])
def test_rows_of_four_and_of_one_have_the_same_bits(dim):
    large = table(70, 30001, dim, "yarn", 16.0, 1.1)
    for at, n in ((0, 1000), (15013, 1), (29001, 1000)):
        assert torch.equal(large[at:at + n], table(70 + at, n, dim, "yarn", 16.0, 1.1))
