"""The scratch memory of the expanded attention: one buffer serves all smaller calls."""

import ctypes
import random

import numpy as np
import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

BF = torch.bfloat16
PART_ROW = (128 + 1) * 4  # bytes of a part's row: 128 results and an lse in fp32


def form(tq, tk, batch, heads, sms=152):
    """item rows, parts, heads of a group, bytes that the call uses, bytes to be allocated"""
    out = [ctypes.c_int() for _ in range(3)] + [ctypes.c_size_t() for _ in range(2)]
    refs = [ctypes.byref(x) for x in out]
    rc = B.load().mla_prefill_form(tq, tk, batch, heads, sms, *refs)
    assert rc == B.MLA_OK, B.load().mla_decode_last_error_string()
    return [x.value for x in out]


def log_int(rng, hi):
    return int(round(hi ** rng.random()))


def sizes(rng):
    return log_int(rng, 20000), log_int(rng, 60000), log_int(rng, 600), log_int(rng, 128)


@pytest.mark.parametrize("sms", [152, 148, 8, 1])
def test_a_larger_call_s_workspace_is_enough(sms):
    rng = random.Random(sms)
    cut = grows = 0
    for _ in range(3000):
        most = sizes(rng)
        given = form(*most, sms)[4]
        assert given <= max(64 << 20, sms * 256 * PART_ROW) and given % 256 == 0
        for _ in range(20):
            less = [rng.choice([n, 1 + rng.randrange(n)]) for n in most]
            rows, parts, group, used, own = form(*less, sms)
            assert rows in (256, 512) and 1 <= parts <= 32 and 1 <= group <= less[3]
            assert used == (0 if parts == 1 else -(-parts * less[0] * less[3] * PART_ROW // 256) * 256)
            assert used <= own <= given
            cut += parts > 1
            grows += used > form(*most, sms)[3]
    assert cut > 100 and grows > 50  # calls that are cut, and smaller ones that use more, are among them


def test_every_number_of_keys():
    """The keys of 200 rows and 60 heads are cut over 600 keys and not over 5000."""
    given = form(200, 5000, 1, 60)[4]
    assert form(200, 5000, 1, 60)[1] == 1 and form(200, 600, 1, 60)[1] == 2
    for tk in range(0, 5001):
        assert form(200, tk, 1, 60)[3] <= given


def test_form_refuses():
    lib, n, b = B.load(), ctypes.byref(ctypes.c_int()), ctypes.byref(ctypes.c_size_t())
    for bad in [(-1, 5, 1, 4, 152), (5, -1, 1, 4, 152), (5, 5, 0, 4, 152), (5, 5, 1, 0, 152), (5, 5, 1, 4, -1), (5, 5, 1, 4, 1 << 17)]:
        assert lib.mla_prefill_form(*bad, n, n, n, b, b) == B.MLA_ERR_ARG
    for i in range(5):
        refs = [n, n, n, b, b]
        refs[i] = None
        assert lib.mla_prefill_form(5, 5, 1, 4, 152, *refs) == B.MLA_ERR_ARG
    assert form(0, 0, 1, 1)[3:] == [0, 0]


@pytest.mark.gpu
def test_one_buffer_for_all_calls():
    """Allocated once for the largest; a smaller call, whose keys are cut where the
    largest one's are not, takes it and gives what its own buffer gives."""
    h = 60
    ws = torch.empty(B.mla_prefill_workspace_bytes(200, 5000, 1, h), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(1)
    q, kv, k_pe = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((200, h, 192), (5000, h, 256), (5000, 64)))
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for tk in (5000, 600, 5000, 300, 600):
        outs = []
        for buffer in (ws, torch.empty(max(256, form(200, tk, 1, h, sms)[3]), dtype=torch.uint8, device="cuda")):
            out, lse = torch.empty(200, h, 128, dtype=BF, device="cuda"), torch.empty(200, h, device="cuda")
            B.mla_prefill(q[..., :128], q[..., 128:], kv[:tk, :, :128], k_pe[:tk], kv[:tk, :, 128:], cu(200), cu(tk), False,
                          1 / np.sqrt(192), out, lse, buffer)
            outs.append((out, lse))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert B.mla_decode_device_error() == 0
    assert form(200, 600, 1, h, 0) == form(200, 600, 1, h, sms)
