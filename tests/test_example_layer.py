"""The example layer, in the library's calls against plain torch.

Both sides round the same quantities to e4m3 (half a step: 2^-4 of a value) and
to bf16; where their fp32 values differ in the last bits, a few codes land on
the other side of a border.  A wrong step (a missed norm, a wrong row, a scale
of another token) is an error of order one.  Bound: one e4m3 half step, 2^-4,
on the norm of the result, and bf16's, 2^-8 with as much again for the codes
that moved, on the residual's."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_layer_step():
    import fp8_layer_step as E

    out, residual = E.main()
    assert out <= 2.0 ** -4 and residual <= 2.0 ** -7
