"""The FP8 products' forms on the host: refusals of the call that makes a product
in a given form, and the choice among them (no GPU is touched by these tests)."""

import ctypes

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


def chosen(t, n, k, experts=1, grouped=False, od=B.MLA_OUT_BF16, out=FAKE, ldo=None, sms=152, clusters=(150, 72, 36)):
    """(tile_tokens, k_parts, copied_results) on a device of 152 SMs, or an error code."""
    res = [ctypes.c_int(-1) for _ in range(3)]
    places = (ctypes.c_int32 * 3)(*clusters) if clusters else None
    rc = B.load().mla_gemm_fp8_form(t, n, k, experts, int(grouped), od, out, n if ldo is None else ldo, sms,
                                    ctypes.addressof(places) if places else None, *[ctypes.byref(r) for r in res])
    return rc if rc else tuple(r.value for r in res)


@pytest.mark.parametrize("args", [
    dict(t=0), dict(t=-1), dict(n=0), dict(k=8), dict(k=24), dict(experts=0, grouped=True), dict(experts=2), dict(ldo=7),
    dict(od=B.MLA_OUT_E4M3), dict(sms=-1), dict(sms=0), dict(clusters=None), dict(t=MOST + 1),
])
def test_form_rejects(args):
    assert chosen(**{**dict(t=4, n=8, k=16), **args}) == B.MLA_ERR_ARG


@pytest.mark.parametrize("od,elt", [(B.MLA_OUT_BF16, 2), (B.MLA_OUT_FP32, 4)])
def test_results_that_the_copy_engine_can_address(od, elt):
    """Its coordinates are 32-bit byte offsets within a row, its row pitch has 40
    bits, and every row starts on 16 bytes: else the warps store the results."""
    def copied(n, **kw):
        form = chosen(8192, n, 512, od=od, **{**dict(ldo=-(-n // 8) * 8), **kw})
        assert form[0] >= 128
        return form[2]

    assert copied(1000) == 1 and copied(1000, out=FAKE + 8) == 0 and copied(1000, ldo=1000 + 8 // elt) == 0
    most = (2 ** 31 - 1) // elt
    assert copied(most) == 1 and copied(most + 1) == 0 and copied(MOST) == 0
    assert copied(1000, ldo=(1 << 40) // elt - 8) == 1 and copied(1000, ldo=(1 << 40) // elt) == 0
    assert chosen(8, 1000, 512, od=od, ldo=1000)[2] == 0  # small tiles are stored by the warps


def test_every_choice_is_a_form_that_is_tested():
    """Over the sizes a layer has, dense and grouped, for several cluster counts:
    the choice is one of the forms that the GPU tests make one by one, and every
    width of tile is somebody's choice."""
    from tests.test_fp8_forms_parity import FORMS

    seen = set()
    for clusters in [(150, 72, 36), (152, 76, 32), (148, 60, 15), (0, 0, 0)]:
        for t in (1, 7, 16, 17, 32, 33, 64, 65, 100, 128, 256, 500, 512, 1024, 4096, 16384):
            for n in (64, 576, 2048, 4096, 7168, 36864):
                for k in (128, 512, 2048, 7168, 16384):
                    seen.add(chosen(t, n, k, clusters=clusters)[:2])
                    for e in (2, 8, 256):
                        seen.add(chosen(t, n, k, e, True, clusters=clusters)[:2])
    assert seen <= set(FORMS) and {tile for tile, _ in seen} == {16, 32, 64, 128, 256}


def test_in_form_valid_arguments_reach_the_device_check():
    if torch.cuda.is_available():
        pytest.skip("valid arguments on fake pointers would launch on a GPU")
    reached = (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)
    for over in [dict(), dict(parts=8), dict(tile=64, parts=4, give_up=7), dict(tile=128), dict(tile=256),
                 dict(off=FAKE, e=3, tile=32, parts=2), dict(give_up=3)]:
        assert call(**over) in reached
    assert call(t=0, a=None, out=None) == B.MLA_OK
