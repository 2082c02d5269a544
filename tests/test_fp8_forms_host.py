"""Refusals of the call that makes an FP8 product in a given form, on the host
(no GPU is touched by these tests)."""

import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

FAKE = 1 << 20  # aligned, non-NULL, never dereferenced


def call(**over):
    kw = dict(a=FAKE, lda=4096, sa=FAKE, ss=4, w=FAKE, ldw=4096, sw=FAKE, off=None, e=1, t=4, n=200, k=4096, out=FAKE,
              od=B.MLA_OUT_BF16, ldo=200, tile=16, parts=1, give_up=-1)
    kw.update(over)
    return B.load().mla_gemm_fp8_in_form(*kw.values(), None)


@pytest.mark.parametrize("over", [
    dict(tile=0), dict(tile=8), dict(tile=48), dict(tile=512), dict(parts=0), dict(parts=3), dict(parts=16),
    dict(tile=128, parts=2), dict(tile=256, parts=2), dict(parts=8, k=1920), dict(parts=2, k=384), dict(give_up=-2),
    dict(give_up=4), dict(tile=32, give_up=8), dict(tile=128, give_up=0), dict(tile=256, give_up=0), dict(e=2),
    dict(off=FAKE, e=0), dict(off=FAKE, e=B.MLA_GEMM_MAX_EXPERTS + 1), dict(lda=4000), dict(k=250), dict(out=None),
    dict(t=1 << 20, ss=1 << 20, n=1 << 21, ldo=1 << 21, parts=2),
])
def test_in_form_rejects(over):
    assert call(**over) == B.MLA_ERR_ARG
    assert B.load().mla_decode_last_error_string()


MOST = 2 ** 31 - 256  # rows are numbered in 32 bits, to the end of a tile of 256 that begins with the last one


@pytest.mark.parametrize("over,fits", [
    (dict(t=MOST, ss=MOST), True), (dict(t=MOST + 1, ss=MOST + 1), False), (dict(t=2 ** 31 - 1, ss=2 ** 31 - 1), False),
    (dict(n=MOST, ldo=MOST, t=1), True), (dict(n=MOST + 1, ldo=MOST + 1, t=1), False),
    (dict(e=8, n=MOST // 8), True), (dict(e=8, n=MOST // 8 + 1), False), (dict(e=1023, n=2 ** 31 // 1023), False),
])
def test_rows_that_32_bits_number(over, fits):
    """Tiles of an expert may begin at any row: the last one's end, past the
    rows, still has to be a positive 32-bit number."""
    lib = B.load()
    kw = dict(a=FAKE, lda=16, sa=FAKE, ss=4, w=FAKE, ldw=16, sw=FAKE, off=FAKE, e=1, t=4, n=8, k=16, out=FAKE,
              od=B.MLA_OUT_FP32, ldo=1 << 32)
    kw.update(over)
    if fits and torch.cuda.is_available():
        pytest.skip("valid arguments on fake pointers would launch on a GPU")
    dense = {k: v for k, v in kw.items() if k not in ("off", "e")}
    calls = [lib.mla_grouped_gemm_fp8(*kw.values(), None)]
    if kw["e"] == 1:
        calls.append(lib.mla_gemm_fp8(*dense.values(), None))
    for rc in calls:
        assert (rc in (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)) if fits else rc == B.MLA_ERR_ARG


def test_in_form_valid_arguments_reach_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("valid arguments on fake pointers would launch on a GPU")
    reached = (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)
    for over in [dict(), dict(parts=8), dict(tile=64, parts=4, give_up=7), dict(tile=128), dict(tile=256),
                 dict(off=FAKE, e=3, tile=32, parts=2), dict(give_up=3)]:
        assert call(**over) in reached
    assert call(t=0, a=None, out=None) == B.MLA_OK
