"""A CUDA error is reported by the call that met it and by no later one."""

import ctypes

import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_a_failed_call_leaves_no_error_for_the_next():
    """Reading the error word synchronises with the default stream, which the
    capture of a stream ordered with it does not allow: that call fails, the ones
    after the capture do not."""
    torch.cuda.init()
    name = "libcudart.so." + torch.version.cuda.split(".")[0]
    rt = ctypes.CDLL(name)
    rt.cudaStreamCreate.argtypes = [ctypes.c_void_p]
    rt.cudaStreamDestroy.argtypes = [ctypes.c_void_p]
    rt.cudaStreamBeginCapture.argtypes = [ctypes.c_void_p, ctypes.c_int]
    rt.cudaStreamEndCapture.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib, x = B.load(), torch.ones(4, 256, device="cuda", dtype=torch.bfloat16)
    w, y = torch.ones(256, device="cuda", dtype=torch.bfloat16), torch.empty_like(x)
    y8, sc = torch.empty(4, 256, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(2, 4, device="cuda")
    rows = torch.zeros(4, 64, device="cuda", dtype=torch.int32)
    index, lens = torch.zeros(4, device="cuda", dtype=torch.int32), torch.ones(4, device="cuda", dtype=torch.int32)
    table = torch.empty(4, 1, device="cuda", dtype=torch.int32)
    calls = [lambda: B.mla_add_rmsnorm(x, None, None, 0, w, 0.0, y, B.MLA_OUT_BF16),
             lambda: B.mla_act_quantize(x, B.MLA_ACT_NONE, y8, B.MLA_OUT_E4M3, sc),
             lambda: B.mla_block_table_from_tokens(rows, index, lens, 64, table)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    stream = ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    for call in calls:
        graph, code = ctypes.c_void_p(), ctypes.c_int()
        assert rt.cudaStreamBeginCapture(stream, 0) == 0  # 0: unsafe calls of any thread are refused
        rc = lib.mla_decode_device_error(ctypes.byref(code), 0)
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        rt.cudaGetLastError()
        assert rc == B.MLA_ERR_CUDA and graph.value is None
        call()
    torch.cuda.synchronize()
    assert rt.cudaStreamDestroy(stream) == 0
    assert B.mla_decode_device_error() == 0
    assert torch.all(y == 1)
