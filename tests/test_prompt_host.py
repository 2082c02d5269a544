"""Refusals of the prompt's operators, on the host: every bad argument is rejected
before any launch (no GPU is touched by these tests)."""

import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

FAKE = 1 << 20  # aligned, non-NULL, never dereferenced
REACHED = (B.MLA_ERR_CUDA, B.MLA_ERR_UNSUPPORTED)  # past the checks, stopped by the missing device
NAN, INF = float("nan"), float("inf")


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("valid arguments on fake pointers would launch on a GPU")


def caller(name, defaults):
    def call(**over):
        assert set(over) <= set(defaults)
        return getattr(B.load(), name)(*{**defaults, **over}.values(), None)
    return call


table = caller("mla_rope_table", dict(t=FAKE, first=0, n=100, dim=64, base=1e4, scaling=B.MLA_ROPE_YARN, factor=40.0,
                                      orig=4096, fast=32.0, slow=1.0, mag=1.0))
rope = caller("mla_rope", dict(q=FAKE, qt=1536, qh=192, k=FAKE, ks=576, t=4, h=8, r=64, pos=FAKE, cs=FAKE, p=100, neox=0,
                               qo=FAKE, qot=512, qoh=64, ko=FAKE, kos=64))
gather = caller("mla_cache_gather", dict(kv=FAKE, kd=B.MLA_KV_E4M3, pages=10, page=64, bt=FAKE, bts=4, starts=FAKE, cu=FAKE,
                                         b=2, t=100, ks=1.0, lat=FAKE, ld=B.MLA_OUT_E4M3, ls=512, sc=FAKE, ss=100, pe=FAKE,
                                         pes=64))
prefill = caller("mla_prefill", dict(qn=FAKE, qnt=1536, qnh=192, qp=FAKE, qpt=1536, qph=192, kn=FAKE, knt=2048, knh=256,
                                     kp=FAKE, kps=64, v=FAKE, vt=2048, vh=256, cq=FAKE, ck=FAKE, b=2, tq=10, tk=20, h=8,
                                     causal=1, scale=0.07, out=FAKE, ot=1024, oh=128, lse=FAKE, ws=None, wsb=0))
merge = caller("mla_merge_states", dict(a=FAKE, at=1024, ah=128, la=FAKE, b=FAKE, bt=1024, bh=128, lb=FAKE, t=4, h=8, d=128,
                                        o=FAKE, ot=1024, oh=128, l=FAKE))

BAD = {
    table: [dict(t=None), dict(t=FAKE + 2), dict(first=-1), dict(n=-1), dict(first=1 << 31, n=1), dict(first=(1 << 31) - 50),
            dict(dim=0), dict(dim=63), dict(dim=B.MLA_ROPE_MAX_DIM + 2), dict(base=1.0), dict(base=NAN), dict(base=INF),
            dict(scaling=3), dict(scaling=-1), dict(factor=0.0), dict(factor=NAN), dict(factor=INF), dict(orig=0),
            dict(slow=0.0), dict(fast=1.0), dict(fast=INF), dict(mag=NAN), dict(mag=1e39),
            dict(scaling=B.MLA_ROPE_LINEAR, factor=-1.0)],
    rope: [dict(t=-1), dict(h=-1), dict(h=65537), dict(r=0), dict(r=7), dict(r=514), dict(p=0), dict(pos=None), dict(cs=None),
           dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(h=0, k=None, ko=None), dict(qt=63), dict(qh=62),
           dict(qot=63), dict(qoh=0), dict(ks=63), dict(kos=1), dict(pos=FAKE + 4), dict(cs=FAKE + 2), dict(q=FAKE + 1),
           dict(qo=FAKE + 1), dict(k=FAKE + 1), dict(ko=FAKE + 1)],
    gather: [dict(kd=2), dict(ld=B.MLA_OUT_FP32), dict(page=16), dict(pages=0), dict(pages=1 << 26), dict(b=0), dict(b=1 << 25),
             dict(bts=0), dict(bts=1 << 31), dict(t=-1), dict(ks=0.0), dict(ks=NAN), dict(ks=INF), dict(kv=None), dict(bt=None),
             dict(cu=None), dict(lat=None), dict(pe=None), dict(sc=None), dict(ls=511), dict(ls=520), dict(pes=60),
             dict(pes=68), dict(ss=99), dict(kv=FAKE + 8), dict(lat=FAKE + 8), dict(pe=FAKE + 2), dict(bt=FAKE + 2),
             dict(starts=FAKE + 1), dict(cu=FAKE + 2), dict(sc=FAKE + 2), dict(ld=B.MLA_OUT_BF16, ls=516)],
    prefill: [dict(tq=-1), dict(tk=-1), dict(tq=(1 << 31) - 1000), dict(tk=(1 << 31) - 1000), dict(b=0), dict(b=1 << 25),
              dict(h=0), dict(h=65537), dict(h=65536, tq=1 << 24, b=1), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN),
              dict(scale=INF), dict(scale=1e-40), dict(qn=None), dict(qp=None), dict(kn=None), dict(kp=None), dict(v=None),
              dict(cq=None), dict(ck=None), dict(out=None), dict(lse=None), dict(qnt=120), dict(qnt=1540), dict(qnh=100),
              dict(qph=56), dict(qpt=1537), dict(knt=2049), dict(knh=127), dict(kps=60), dict(kps=72 + 4), dict(vt=64),
              dict(vh=132), dict(ot=1020), dict(oh=64), dict(knt=1 << 39), dict(qn=FAKE + 8), dict(qp=FAKE + 2),
              dict(kn=FAKE + 4), dict(kp=FAKE + 8), dict(v=FAKE + 8), dict(out=FAKE + 8), dict(lse=FAKE + 2),
              dict(cq=FAKE + 2), dict(ck=FAKE + 1)],
    merge: [dict(t=-1), dict(h=0), dict(h=65537), dict(d=0), dict(d=4), dict(d=132), dict(d=B.MLA_MERGE_MAX_DIM + 8),
            dict(t=1 << 20, h=1 << 12), dict(a=None), dict(la=None), dict(b=None), dict(lb=None), dict(o=None), dict(l=None),
            dict(at=120), dict(ah=64), dict(bt=1028), dict(bh=0), dict(ot=4), dict(oh=132), dict(a=FAKE + 8), dict(b=FAKE + 2),
            dict(o=FAKE + 8), dict(la=FAKE + 1), dict(lb=FAKE + 2), dict(l=FAKE + 2)],
}


@pytest.mark.parametrize("f,over", [(f, o) for f, os in BAD.items() for o in os], ids=str)
def test_rejects(f, over):
    assert f(**over) == B.MLA_ERR_ARG
    assert B.load().mla_decode_last_error_string()


def test_no_tokens_is_a_no_op():
    assert table(n=0, t=None) == B.MLA_OK
    assert rope(t=0, q=None, k=None, pos=None) == B.MLA_OK
    assert gather(t=0, kv=None, lat=None) == B.MLA_OK
    assert prefill(tq=0, qn=None, out=None, tk=5) == B.MLA_OK
    assert merge(t=0, a=None, o=None) == B.MLA_OK


def test_valid_arguments_reach_the_device_check():
    no_gpu()
    assert table() in REACHED and table(scaling=B.MLA_ROPE_PLAIN, factor=NAN, orig=0, fast=0.0) in REACHED
    assert table(first=(1 << 31) - 100) in REACHED and table(dim=2) in REACHED
    assert rope() in REACHED and rope(k=None, ko=None, ks=0) in REACHED and rope(h=0, q=None, qo=None) in REACHED
    assert rope(q=FAKE + 2, r=6, qt=7, qh=7, h=1) in REACHED and rope(h=1, qh=0, qoh=-3) in REACHED
    assert gather() in REACHED and gather(starts=None) in REACHED and gather(kd=B.MLA_KV_BF16, ks=0.0) in REACHED
    assert gather(ld=B.MLA_OUT_BF16, sc=None, ss=0) in REACHED
    assert prefill() in REACHED and prefill(tk=0, kn=None, kp=None, v=None, knt=0) in REACHED
    assert prefill(h=1, qnh=0, vh=-5, oh=1) in REACHED and prefill(causal=0) in REACHED
    assert merge() in REACHED and merge(h=1, ah=0, bh=-8, oh=0) in REACHED and merge(d=72) in REACHED


def test_binding_checks_tensors():
    """The binding refuses what the C call cannot see: shapes, types, host memory."""
    def bad(f, *args, **kw):
        with pytest.raises(B.MlaError) as e:
            f(*args, **kw)
        assert e.value.code == B.MLA_ERR_ARG

    bf, i32 = torch.bfloat16, torch.int32
    bad(B.mla_rope_table, torch.zeros(4, 64))                       # host memory
    q, k, pos, cs = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, 64, dtype=bf), torch.zeros(4, dtype=torch.long), torch.zeros(9, 64)
    for args in [(q, k, pos, cs, False, q, k), (q, k, pos.int(), cs, False, q, k), (q.float(), k, pos, cs, False, q, k),
                 (q[:3], k, pos, cs, False, q, k), (q, None, pos, cs, False, q, k), (q, k, pos, cs[:, :32], False, q, k)]:
        bad(B.mla_rope, *args)
    kv, bt, cu_, lat, pe = (torch.zeros(3, 64, 576, dtype=bf), torch.zeros(2, 3, dtype=i32), torch.zeros(3, dtype=i32),
                            torch.zeros(5, 512, dtype=bf), torch.zeros(5, 64, dtype=bf))
    for args in [(kv, B.MLA_KV_BF16, bt, None, cu_, 1.0, lat, B.MLA_OUT_BF16, None, pe),
                 (kv, B.MLA_KV_E4M3, bt, None, cu_, 1.0, lat, B.MLA_OUT_BF16, None, pe),
                 (kv, B.MLA_KV_BF16, bt, cu_, cu_, 1.0, lat, B.MLA_OUT_BF16, None, pe),
                 (kv, B.MLA_KV_BF16, bt, None, cu_[:2], 1.0, lat, B.MLA_OUT_BF16, None, pe),
                 (kv, B.MLA_KV_BF16, bt, None, cu_, 1.0, lat[:, :500], B.MLA_OUT_BF16, None, pe)]:
        bad(B.mla_cache_gather, *args)
    qn, qp, kn, v, out = (torch.zeros(4, 2, d, dtype=bf) for d in (128, 64, 128, 128, 128))
    lse, c2 = torch.zeros(4, 2), torch.zeros(2, dtype=i32)
    good = [qn, qp, kn, k, v, c2, c2, True, 0.07, out, lse]
    bad(B.mla_prefill, *good)                                       # host memory
    for i, x in [(1, qn), (2, kn[:, :1]), (3, k[:3]), (4, v.float()), (5, c2.long()), (6, cu_), (9, out[:3]), (10, lse.t())]:
        bad(B.mla_prefill, *good[:i], x, *good[i + 1:])
    bad(B.mla_merge_states, out, lse, out, lse, out, lse)           # host memory
    bad(B.mla_merge_states, out, lse, out, lse, out[:, :1], lse)
