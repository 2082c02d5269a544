"""Refusals of the FP8 layer operators, on the host: every bad argument is
rejected before any launch (no GPU is touched by these tests)."""

import numpy as np
import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

FAKE = 1 << 20  # aligned, non-NULL, never dereferenced


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("valid arguments on fake pointers would launch on a GPU")


REACHED = (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)  # past the checks, stopped by the missing device


def call_norm(**over):
    kw = dict(x=FAKE, xs=256, ri=FAKE, ro=FAKE, rd=B.MLA_OUT_BF16, rs=256, w=FAKE, t=4, d=256, eps=1e-6, y=FAKE,
              yd=B.MLA_OUT_E4M3, ys=256, sc=FAKE, ss=4)
    kw.update(over)
    return B.load().mla_add_rmsnorm(*kw.values(), None)


@pytest.mark.parametrize("over", [
    dict(t=-1), dict(d=0), dict(d=B.MLA_NORM_MAX_DIM + 1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(x=None), dict(w=None), dict(y=None), dict(x=FAKE + 1), dict(w=FAKE + 1),
    dict(xs=255), dict(ri=None), dict(ro=None), dict(rd=B.MLA_OUT_E4M3), dict(rs=255), dict(ri=FAKE + 1),
    dict(rd=B.MLA_OUT_FP32, ro=FAKE + 2), dict(yd=B.MLA_OUT_FP32), dict(ys=255), dict(sc=None), dict(sc=FAKE + 2),
    dict(ss=3), dict(yd=B.MLA_OUT_BF16, y=FAKE + 1),
])
def test_norm_rejects(over):
    assert call_norm(**over) == B.MLA_ERR_ARG
    assert B.load().mla_decode_last_error_string()


def call_act(**over):
    kw = dict(x=FAKE, xs=512, act=B.MLA_ACT_SILU_MUL, t=4, d=256, y=FAKE, yd=B.MLA_OUT_E4M3, ys=256, sc=FAKE, ss=4)
    kw.update(over)
    return B.load().mla_act_quantize(*kw.values(), None)


@pytest.mark.parametrize("over", [
    dict(act=2), dict(t=-1), dict(d=0), dict(d=1 << 30), dict(t=1 << 30), dict(x=None), dict(x=FAKE + 1), dict(xs=511),
    dict(act=B.MLA_ACT_NONE, yd=B.MLA_OUT_BF16), dict(y=None), dict(yd=B.MLA_OUT_FP32), dict(ys=255), dict(sc=None),
    dict(sc=FAKE + 1), dict(ss=3),
])
def test_act_rejects(over):
    assert call_act(**over) == B.MLA_ERR_ARG


GEMM = dict(a=FAKE, lda=256, sa=FAKE, ss=4, w=FAKE, ldw=256, sw=FAKE)
REST = dict(t=4, n=200, k=256, out=FAKE, od=B.MLA_OUT_BF16, ldo=200)
GEMM_BAD = [
    dict(t=-1), dict(n=0), dict(k=0), dict(k=8), dict(k=250), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None),
    dict(out=None), dict(lda=240), dict(lda=264), dict(ldw=240), dict(ldw=257), dict(lda=1 << 40), dict(ldw=1 << 41),
    dict(ss=3), dict(ldo=199), dict(od=B.MLA_OUT_E4M3), dict(od=9), dict(a=FAKE + 8), dict(w=FAKE + 8),
    dict(sa=FAKE + 2), dict(sw=FAKE + 1), dict(out=FAKE + 1), dict(od=B.MLA_OUT_FP32, out=FAKE + 2),
]


def call_gemm(**over):
    return B.load().mla_gemm_fp8(*{**GEMM, **REST, **over}.values(), None)


def call_grouped(**over):
    return B.load().mla_grouped_gemm_fp8(*{**GEMM, "off": FAKE, "e": 3, **REST, **over}.values(), None)


@pytest.mark.parametrize("over", GEMM_BAD)
def test_gemm_rejects(over):
    assert call_gemm(**over) == B.MLA_ERR_ARG
    assert B.load().mla_decode_last_error_string()


@pytest.mark.parametrize("over", GEMM_BAD + [
    dict(off=None), dict(off=FAKE + 2), dict(e=0), dict(e=B.MLA_GEMM_MAX_EXPERTS + 1), dict(e=1024, n=1 << 21),
])
def test_grouped_gemm_rejects(over):
    assert call_grouped(**over) == B.MLA_ERR_ARG


def test_no_tokens_is_a_no_op():
    assert call_norm(t=0, x=None, y=None, sc=None) == B.MLA_OK
    assert call_act(t=0, x=None, y=None, sc=None) == B.MLA_OK
    assert call_gemm(t=0, a=None, sa=None, out=None) == B.MLA_OK
    assert call_grouped(t=0, a=None, sa=None, out=None) == B.MLA_OK


def test_valid_arguments_reach_the_device_check():
    no_gpu()
    assert call_norm() in REACHED
    assert call_norm(ri=None, ro=None, rd=77, rs=0) in REACHED       # no residual: its type and stride are unused
    assert call_norm(yd=B.MLA_OUT_BF16, sc=None, ss=0) in REACHED    # a bf16 result has no scales
    assert call_norm(d=7, xs=9, ys=7, rs=7, x=FAKE + 2, y=FAKE + 1) in REACHED
    assert call_act() in REACHED and call_act(act=B.MLA_ACT_NONE, xs=256) in REACHED
    assert call_act(yd=B.MLA_OUT_BF16, sc=None, ss=0) in REACHED
    assert call_gemm() in REACHED and call_gemm(k=16, n=1, od=B.MLA_OUT_FP32) in REACHED
    assert call_grouped() in REACHED


def test_binding_checks_tensors():
    """The binding refuses what the C call cannot see: shapes, types, host memory."""
    def bad(f, *args):
        with pytest.raises(B.MlaError) as e:
            f(*args)
        assert e.value.code == B.MLA_ERR_ARG

    f8, bf, f32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
    x, w, y, sc = torch.zeros(4, 256, dtype=bf), torch.zeros(256, dtype=bf), torch.zeros(4, 256, dtype=f8), torch.zeros(2, 4)
    for args in [(x, None, None, 0, w, 1e-6, y, B.MLA_OUT_E4M3, sc),                    # host memory
                 (x.half(), None, None, 0, w, 1e-6, y, B.MLA_OUT_E4M3, sc),             # fp16 is not bf16
                 (x, None, None, 0, w, 1e-6, y[:3], B.MLA_OUT_E4M3, sc),
                 (x, None, None, 0, w[:255], 1e-6, y, B.MLA_OUT_E4M3, sc),
                 (x, None, None, 0, w, 1e-6, y, B.MLA_OUT_E4M3, sc.t()),
                 (x.t(), None, None, 0, w, 1e-6, y, B.MLA_OUT_E4M3, sc)]:
        bad(B.mla_add_rmsnorm, *args)
    bad(B.mla_act_quantize, x, B.MLA_ACT_SILU_MUL, y, B.MLA_OUT_E4M3, sc)               # x must be twice as wide
    bad(B.mla_act_quantize, x, B.MLA_ACT_NONE, y, B.MLA_OUT_E4M3, sc)
    a, b, sb, out = y, torch.zeros(200, 256, dtype=f8), torch.zeros(2, 2), torch.zeros(4, 200, dtype=f32)
    bad(B.mla_gemm_fp8, a, sc, b, sb, out, B.MLA_OUT_FP32)                              # host memory
    bad(B.mla_gemm_fp8, a, sc, b[:, :240], sb, out, B.MLA_OUT_FP32)
    bad(B.mla_gemm_fp8, a.to(torch.float8_e5m2), sc, b, sb, out, B.MLA_OUT_FP32)
    bad(B.mla_gemm_fp8, a, sc, b, sb, out, B.MLA_OUT_BF16)                              # type and code differ
    off = torch.zeros(4, dtype=torch.int32)
    bad(B.mla_grouped_gemm_fp8, a, sc, b, sb, off, out, B.MLA_OUT_FP32)                 # w is 2-D
    w3, s3 = torch.zeros(3, 200, 256, dtype=f8), torch.zeros(3, 2, 2)
    bad(B.mla_grouped_gemm_fp8, a, sc, w3, s3, off, out, B.MLA_OUT_FP32)
    bad(B.mla_grouped_gemm_fp8, a, sc, w3.transpose(0, 1), s3, off, out, B.MLA_OUT_FP32)
    assert np.all(out.numpy() == 0)
