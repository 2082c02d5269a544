"""Expanded attention where a CTA takes many items whose tiles are uneven: rows that
see no key, requests of one step among longer ones, requests without a row between;
heads in groups; more items than clusters."""

import ctypes

import numpy as np
import pytest
import torch

from paged_mla_decode_08_gb300 import binding as B

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SCALE = 1 / np.sqrt(192)


@pytest.fixture(autouse=True)
def no_device_error():
    B.mla_decode_device_error(reset=True)
    yield
    assert B.mla_decode_device_error(reset=True) == 0


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF)


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Call:
    def __init__(self, h, q_lens, k_lens, causal, seed=1):
        self.q_lens, self.k_lens, self.causal, self.h = list(map(int, q_lens)), list(map(int, k_lens)), causal, h
        self.tq, self.tk = sum(self.q_lens), sum(self.k_lens)
        self.q, self.kv, self.k_pe = randn(self.tq, h, 192, seed=seed), randn(self.tk, h, 256, seed=seed + 1), randn(self.tk, 64, seed=seed + 2)
        self.cq, self.ck = cu(self.q_lens), cu(self.k_lens)
        need = B.mla_prefill_workspace_bytes(self.tq, self.tk, len(self.q_lens), h)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None

    def run(self):
        out = torch.full((self.tq, self.h, 128), 7, dtype=BF, device="cuda")
        lse = torch.full((self.tq, self.h), 7.0, device="cuda")
        B.mla_prefill(self.q[..., :128], self.q[..., 128:], self.kv[..., :128], self.k_pe, self.kv[..., 128:], self.cq, self.ck,
                      self.causal, SCALE, out, lse, self.ws)
        return out, lse

    def check(self, out, lse, heads=None):
        """fp64, over some heads of every request.  What is allowed: 2^-8 of the weights'
        mass for weights rounded to bf16, as much again for scores (192 fp32 products,
        24 additions off by 2^-22 of sum |q k| scale, below 40 here: 2^-12, twice) and fp32
        sums, and 2^-8 of the result for its rounding.  An lse moves by the score's 2^-12 and
        its own few steps of 2^-24 of at most 16."""
        heads = list(range(self.h)) if heads is None else heads
        q0 = k0 = 0
        for n, m in zip(self.q_lens, self.k_lens):
            if n:
                k = torch.cat([self.kv[k0:k0 + m, heads, :128], self.k_pe[k0:k0 + m, None].expand(-1, len(heads), -1)], -1).double()
                v = self.kv[k0:k0 + m, heads, 128:].double()
                s = SCALE * torch.einsum("qhd,khd->hqk", self.q[q0:q0 + n, heads].double(), k)
                if self.causal:
                    s.masked_fill_(torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None], -float("inf"))
                some = torch.arange(n, device="cuda") >= (n - m if self.causal else 0) if m else torch.zeros(n, dtype=torch.bool, device="cuda")
                got, got_lse = out[q0:q0 + n, heads], lse[q0:q0 + n, heads]
                assert not got[~some].any() and torch.all(got_lse[~some] == -float("inf"))
                s = s[:, some]
                w = torch.softmax(s, -1)
                want, mass = torch.einsum("hqk,khd->qhd", w, v), torch.einsum("hqk,khd->qhd", w, v.abs())
                assert torch.all((got[some].double() - want).abs() <= 2.0 ** -7 * mass + 2.0 ** -8 * want.abs())
                if some.any():
                    assert torch.all((got_lse[some].double() - torch.logsumexp(s, -1).T).abs() <= 2.0 ** -11)
            q0, k0 = q0 + n, k0 + m


def between(q_lens, k_lens, gap):
    """A request without a row, of `gap` keys, behind each: its keys are no one's."""
    q, k = [], []
    for n, m in zip(q_lens, k_lens):
        q += [n, 0]
        k += [m, gap]
    return q, k


# What a tile's warps may come to while the other tile's values are still on their way:
# several items in which a tile has no step, then one in which both look values through.
SHORT = [60, 50, 33]                                       # one step on one CTA: the second tile has none
UNEVEN = {
    "short then two steps": (152, (SHORT + [120]) * 6, (SHORT + [150]) * 6),
    "short then three steps": (152, (SHORT + [128, 9]) * 6, (SHORT + [190, 64]) * 6),
    "rows without a key": (152, [256, 256, 256, 256, 100] * 6, [100, 128, 60, 400, 130] * 6),
    "rows without a key, several blocks": (76, [700, 300, 513] * 6, [130, 40, 520] * 6),
    "in pairs": (19, [600, 900, 512, 520, 513] * 5, [130, 2900, 200, 2500, 700] * 5),
}


@pytest.mark.parametrize("name", UNEVEN)
def test_tiles_that_run_ahead(name):
    """Keys and values that no row sees may hold anything, whatever the other tile of the
    CTA is at: the results keep their bits, run after run."""
    h, q_lens, k_lens = UNEVEN[name]
    c = Call(h, *between(q_lens, k_lens, 70), True)
    assert (form(c)[0] == 512) == (name == "in pairs")
    clean = c.run()
    c.check(*clean, heads=[0, h // 2, h - 1])
    ends = c.ck.tolist()
    for b in range(1, len(c.q_lens), 2):
        c.kv[ends[b]:ends[b + 1]] = (float("nan"), float("inf"), -float("inf"))[b // 2 % 3]
        c.k_pe[ends[b]:ends[b + 1]] = float("nan")
    for _ in range(20):
        again = c.run()
        assert torch.equal(again[0], clean[0]) and torch.equal(again[1], clean[1])


def form(c):
    out = [ctypes.c_int() for _ in range(3)] + [ctypes.c_size_t() for _ in range(2)]
    assert B.load().mla_prefill_form(c.tq, c.tk, len(c.q_lens), c.h, 0, *map(ctypes.byref, out)) == B.MLA_OK
    return [x.value for x in out[:3]]


def blocks(lens, item_rows):
    return sum(-(-n // item_rows) for n in lens)


GROUPS = [  # heads, rows, keys, item rows, whether the keys are cut
    (19, [1000], [8192], 512, True), (19, [100], [8192], 256, True), (37, [3000], [3000], 512, False),
    (71, [60, 90, 256, 31], [4000, 4100, 256, 9000], 256, False), (151, [40] * 40, [1500, 600] * 20, 256, False),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("h, q_lens, k_lens, item_rows, cut", GROUPS)
def test_heads_in_groups(h, q_lens, k_lens, item_rows, cut, causal):
    """Heads whose number their group's does not divide, in both forms, in parts and
    with more requests than a warp has lanes."""
    c = Call(h, q_lens, k_lens, causal)
    rows, parts, group = form(c)
    assert rows == item_rows and (parts > 1) == cut and group < h and h % group
    c.check(*c.run(), heads=sorted({0, group - 1, group, h - 1}))


def test_pairs_of_more_requests_than_lanes():
    c = Call(3, [140] * 40, [700 + 5 * i for i in range(40)], True)
    assert form(c)[0] == 512
    c.check(*c.run())


def test_pairs_with_more_items_than_clusters():
    """Clusters go on by their number before they ask for another's items."""
    rng = np.random.default_rng(5)
    q_lens = np.where(rng.random(170) < 0.1, 0, rng.integers(140, 230, 170))
    c = Call(8, q_lens, rng.integers(610, 760, 170), True)
    rows, parts, _ = form(c)
    clusters = max(2 * -(-c.tq // rows) * c.h * parts, 8 * torch.cuda.get_device_properties(0).multi_processor_count // 2)
    assert rows == 512 and blocks(c.q_lens, rows) * c.h > clusters
    c.check(*c.run(), heads=[0, 5, 7])


@pytest.mark.parametrize("h, q_lens, k_lens, item_rows", [
    (16, [120] * 4, [130, 4000, 130, 140], 256), (16, [200] * 4, [6000, 700, 300, 1000], 512), (50, [1, 255, 2, 100], [3000, 300, 1, 90], 256)])
def test_parts_of_more_rows_than_the_merge_takes_at_once(h, q_lens, k_lens, item_rows):
    """Its CTAs go on to their block's next rows; requests that are not cut lie between."""
    c = Call(h, q_lens, k_lens, True)
    rows, parts, _ = form(c)
    groups, at_once = rows // 8, 8 * torch.cuda.get_device_properties(0).multi_processor_count
    assert rows == item_rows and parts > 1 and blocks(q_lens, rows) * h * groups > at_once
    out, lse = c.run()
    c.check(out, lse, heads=[0, 1, h - 1])
    assert all(torch.equal(a, b) for a, b in zip(c.run(), (out, lse)))


def test_few_keys_are_not_cut_for_one_request_alone():
    """Even requests of few keys have no second launch."""
    assert form(Call(16, [130] * 4, [130] * 4, True))[1] == 1
    assert form(Call(16, [130] * 4, [130, 1200, 130, 130], True))[1] > 1
