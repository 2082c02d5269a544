"""What the prompt's operators read may be results of the kernel before, which can still
run while they are resident: offsets, first tokens and block tables among them.  The
combine stands to the main kernel, whose partials it reads, in the same way."""

import os
import re

import numpy as np
import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B
from paged_mla_decode_08_gb300 import build

BF = torch.bfloat16
SCALE = 1 / np.sqrt(192)


@pytest.mark.parametrize("source", ["mla_prefill.cu", "mla_prompt_rows.cu", "mla_combine.cu"])
def test_no_read_only_loads(source):
    """They promise that nobody writes the data in the kernel's lifetime, which begins
    before the kernel before it has ended."""
    with open(os.path.join(os.path.dirname(build.__file__), "csrc", source)) as f:
        code = re.sub(r"//.*", "", f.read())
    assert "griddepcontrol.wait" in code
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc\b|__restrict__", code)


class Late:
    """int32 numbers that a long kernel writes last: the last row of a norm's residual
    output (0 + bits, exact)."""

    def __init__(self, count):
        self.source = torch.zeros(20000, count, device="cuda")
        self.x, self.written = torch.zeros(20000, count, dtype=BF, device="cuda"), torch.zeros_like(self.source)
        self.weight, self.y = torch.ones(count, dtype=BF, device="cuda"), torch.empty_like(self.x)
        self.numbers = self.written[-1].view(torch.int32)

    def set(self, values):
        self.source[-1].view(torch.int32).copy_(torch.from_numpy(np.asarray(values, dtype=np.int32)))

    def write(self):
        B.mla_add_rmsnorm(self.x, self.source, self.written, B.MLA_OUT_FP32, self.weight, 1.0, self.y, B.MLA_OUT_BF16)


def rounds(late, values, step, outs, again):
    """Call by call and replayed, against a call whose numbers were there long before."""
    late.set(values(0))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        now = np.asarray(values(i), dtype=np.int32)
        late.set(now)
        for x in outs:
            x.view(torch.uint8).fill_(9)
        torch.cuda.synchronize()
        graph.replay() if i % 2 else step()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for x in outs:
            x.view(torch.uint8).fill_(9)
        numbers = torch.from_numpy(now).cuda()
        torch.cuda.synchronize()
        again(numbers)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, outs))
    assert B.mla_decode_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("h, batch, tq, tk", [(4, 5, 300, 900), (4, 5, 2000, 6000), (2, 3, 100, 9000), (3, 70, 900, 2000)])
def test_offsets_of_the_attention(h, batch, tq, tk):
    """One CTA an item, pairs, parts with their merge, more requests than a warp has lanes."""
    B.mla_decode_device_error(reset=True)
    g = torch.Generator().manual_seed(tq)
    rand = lambda *shape: torch.randn(*shape, generator=g).to(BF).cuda()  # noqa: E731
    q, kv, k_pe = rand(tq, h, 192), rand(tk, h, 256), rand(tk, 64)
    out, lse = torch.empty(tq, h, 128, dtype=BF, device="cuda"), torch.empty(tq, h, device="cuda")
    need = B.mla_prefill_workspace_bytes(tq, tk, batch, h)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    late = Late(2 * (batch + 1))

    def values(i):
        rng = np.random.default_rng(100 * batch + i)
        return np.concatenate([np.sort(np.concatenate([[0, n], rng.integers(0, n + 1, batch - 1)])) for n in (tq, tk)])

    def attend(cq, ck):
        B.mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], k_pe, kv[..., 128:], cq, ck, False, SCALE, out, lse, ws)

    def step():
        late.write()
        attend(late.numbers[:batch + 1], late.numbers[batch + 1:])

    rounds(late, values, step, (out, lse), lambda n: attend(n[:batch + 1], n[batch + 1:]))


@pytest.mark.gpu
@pytest.mark.parametrize("batch, tokens", [(3, 50), (40, 1000), (300, 600)])
def test_offsets_starts_and_block_table_of_the_gather(batch, tokens):
    B.mla_decode_device_error(reset=True)
    width, pages = tokens // 64 + 3, 50
    kv = torch.randn(pages, 64, 576, generator=torch.Generator().manual_seed(batch)).to(BF).cuda()
    rows, pe = torch.empty(tokens, 512, dtype=BF, device="cuda"), torch.empty(tokens, 64, dtype=BF, device="cuda")
    late = Late(batch + 1 + batch + batch * width)

    def values(i):
        rng = np.random.default_rng(100 * batch + i)
        cu = np.sort(np.concatenate([[0, tokens], rng.integers(0, tokens + 1, batch - 1)]))
        return np.concatenate([cu, rng.integers(0, 64, batch), rng.integers(0, pages, batch * width)])

    def gather(n):
        B.mla_cache_gather(kv, B.MLA_KV_BF16, n[2 * batch + 1:].view(batch, width), n[batch + 1:2 * batch + 1], n[:batch + 1], 1.0,
                           rows, B.MLA_OUT_BF16, None, pe)

    def step():
        late.write()
        gather(late.numbers)

    rounds(late, values, step, (rows, pe), gather)
