"""The FP8 layer operators in a graph, after nodes that are no kernels of theirs:
copies, fills and joins of streams.  Each call is launched as a programmatic
dependent of the work before it, whatever that is; a replay has to give the bits of
the calls made one by one."""

import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_error():
    B.mla_decode_device_error(reset=True)
    yield
    assert B.mla_decode_device_error(reset=True) == 0


def codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g).float().cuda()


@pytest.mark.parametrize("t", [3, 100, 700])
def test_replay_equals_calls_one_by_one(t):
    d, n = 2048, 512
    source, x = codes((t, 2 * d), t).bfloat16(), torch.empty(t, 2 * d, dtype=torch.bfloat16, device="cuda")
    w, sw = codes((2, n, d), 1).to(torch.float8_e4m3fn), torch.rand(2, 4, 16, device="cuda")
    weight = codes((d,), 2).bfloat16()
    act, act_s = torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(16, t, device="cuda")
    y, y_s = torch.empty_like(act), torch.empty_like(act_s)
    out, out2 = torch.empty(t, n, device="cuda"), torch.empty(t, n, device="cuda")
    off_source = torch.tensor([0, t // 3, t], dtype=torch.int32, device="cuda")
    off = torch.zeros_like(off_source)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        x.copy_(source)                                             # a copy before the kernels that read it
        side.wait_stream(main)
        B.mla_act_quantize(x, B.MLA_ACT_SILU_MUL, act, B.MLA_OUT_E4M3, act_s)
        with torch.cuda.stream(side):                               # the norm beside it
            B.mla_add_rmsnorm(x[:, :d], None, None, 0, weight, 1e-6, y, B.MLA_OUT_E4M3, y_s)
        main.wait_stream(side)
        out.zero_()                                                 # a fill and a copy between the kernels
        off.copy_(off_source)
        B.mla_grouped_gemm_fp8(act, act_s, w, sw, off, out, B.MLA_OUT_FP32)
        B.mla_gemm_fp8(y, y_s, w[1], sw[1], out2, B.MLA_OUT_FP32)
        out.add_(out2)                                              # and a kernel that is no dependent of ours

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        source.copy_(codes((t, 2 * d), t + i + 10).bfloat16())
        off_source[1] = (i * t) // 3
        step()
        torch.cuda.synchronize()
        want = [v.view(torch.uint8).clone() for v in (act, act_s, y, y_s, out, out2)]
        for v in (act, act_s, y, y_s, out, out2):
            v.view(torch.uint8).fill_(0x11)
        x.zero_()
        off.zero_()
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, v.view(torch.uint8)) for a, v in zip(want, (act, act_s, y, y_s, out, out2)))
