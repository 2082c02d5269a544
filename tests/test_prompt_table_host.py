"""Frequencies of the rotary table that are no numbers are refused on the host."""

import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

FAKE = 1 << 20  # aligned, non-NULL, never dereferenced


def call(scaling, factor, dim=64, base=1e4):
    return B.load().mla_rope_table(FAKE, 0, 100, dim, base, scaling, factor, 4096, 32.0, 1.0, 1.0, None)


@pytest.mark.parametrize("scaling", [B.MLA_ROPE_LINEAR, B.MLA_ROPE_YARN])
@pytest.mark.parametrize("factor", [1e-310, 5e-324])
def test_a_factor_that_overflows_a_frequency(scaling, factor):
    """1 / factor passes the largest double (with YaRN also times a share of 0: NaN); as a
    whole number of turns it would be anything."""
    assert call(scaling, factor) == B.MLA_ERR_ARG
    assert b"finite" in B.load().mla_decode_last_error_string()


def test_small_factors_that_do_not():
    if torch.cuda.is_available():
        pytest.skip("valid arguments on fake pointers would launch on a GPU")
    for factor in (1e-300, 1e-3):
        assert call(B.MLA_ROPE_LINEAR, factor) in (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)
        assert call(B.MLA_ROPE_YARN, factor) in (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)
    assert call(B.MLA_ROPE_PLAIN, 1e-310) in (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)
