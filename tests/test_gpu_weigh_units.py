"""pn_kv_weigh where blocks and warps have many units of work, and where its waits give up.

Keys are whole numbers -8 .. 7 times 2^-10, queries whole numbers, so scores are exact in
fp32 in any order of their sums, and only the exponent's arithmetic errs.  With u = 2^-24,
x the score and l the row's log sum: the argument x f + less errs by u |x - l| where it
is rounded, by u |l| where less is, by u |x - l| for f's own rounding (which the row's
constant makes up for at x = l); ex2 by 2^-22, and the row's constant and its products by
less than 8 u.  So a probability errs by
  2^-22 + 2 u |x - l| + u |l| + 8 u
of itself, and a sum of them over n rows by a chain of n / 4 + 12 additions more.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


class Case:
    """Requests whose tokens lie on pages of their own in any order; some pages of the cache hold nothing."""

    def __init__(self, pn, lens, counts, heads, kv, D, page, window=0, sinks=0, seed=0, cancel=False):
        g = torch.Generator(device="cuda").manual_seed(seed + D + sum(lens))
        self.lens, self.counts, self.group, self.kv, self.page, self.window, self.sinks = lens, counts, heads // kv, kv, page, window, sinks
        held = [-(-n // page) for n in lens]
        pages = sum(held) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        self.table = torch.full((len(lens), max(held) + 1), 1 << 30, dtype=torch.int32, device="cuda")
        at, slots = 0, []
        for b, n in enumerate(lens):
            own = order[at:at + held[b]]
            at += held[b]
            self.table[b, :held[b]] = own.int()
            t = torch.arange(n, device="cuda")
            slots.append(own[t // page] * page + t % page)
        self.slots = slots
        self.cache = pn.kv_cache(pages, page, kv, D)
        self.keys = []
        for s in slots:                                      # every group holds -8, its largest: its scale is 2^-10
            n = torch.randint(-8, 8, (len(s), kv, D), generator=g, device="cuda").float()
            n[:, :, ::64] = -8
            if cancel:
                n[:, :, 40::64] = n[:, :, 1::64]
            pn.kv_append(None, n * 2.0 ** -10, n * 2.0 ** -10, self.cache, s)
            self.keys.append(n.double() * 2.0 ** -10)
        if len(slots[0]):
            assert torch.equal(pn.kv_read(self.cache, slots[0])[0].double(), self.keys[0])
        self.scale = 0.5 if D <= 128 else 0.25                # scores of some units
        self.q = torch.randint(-255, 256, (sum(counts), heads, D), generator=g, device="cuda").half()
        if cancel:
            self.q[:, :, 1::64], self.q[:, :, 40::64] = 2.0 ** 15, -2.0 ** 15
        self.starts = torch.tensor([0, *counts], device="cuda").cumsum(0).int()
        self.device_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.weights = torch.rand(pages, kv, page, generator=g, device="cuda")
        self.most = max(max(counts), 1)
        self.reckon()

    def reckon(self, decay=0.9):
        """log sums, what is expected, and how far from it a call may be."""
        decay = float(torch.tensor(decay))
        self.lse = torch.full(self.q.shape[:2], -math.inf, device="cuda")
        self.want = torch.full(self.weights.shape, -3.0, dtype=torch.float64, device="cuda")
        self.limit = torch.zeros_like(self.want)
        start = 0
        for b, (n, L) in enumerate(zip(self.counts, self.lens)):
            if n and L:
                t, p = torch.arange(L, device="cuda"), L - n + torch.arange(n, device="cuda")
                see = t[:, None] <= p
                if self.window:
                    see &= (t[:, None] > p - self.window) | (t[:, None] < self.sinks)
                slots = self.slots[b]
                for h in range(self.kv):
                    total = torch.zeros(L, dtype=torch.float64, device="cuda")
                    bound = torch.zeros_like(total)
                    for i in range(self.group):
                        row = h * self.group + i
                        x = self.scale * (self.keys[b][:, h] @ self.q[start:start + n, row].double().T)          # [L][n]
                        x = torch.where(see, x, -math.inf)
                        z = torch.logsumexp(x, 0).float()
                        self.lse[start:start + n, row] = z
                        z = z.double()
                        prob = torch.where(see, torch.exp(x - z), 0.0)
                        off = 2.0 ** -22 + 2 * U * (x - z).abs() + U * z.abs() + 8 * U
                        total += prob.sum(1)
                        bound += torch.where(prob > 0, prob * off, 0.0).sum(1)
                    bound += total * (n * self.group / 4 + 12) * U
                    at = (slots // self.page, torch.full_like(slots, h), slots % self.page)
                    before = torch.where(t < L - n, decay * self.weights[at].double(), 0.0)
                    self.want[at] = before + total
                    self.limit[at] = bound + 2 * U * (2 * before + total) + 1e-37
            start += n

    def call(self, pn, decay=0.9, weights=None, out=None):
        return pn.kv_weigh(self.q, self.cache, self.table, self.device_lens, self.starts, self.most, self.lse, self.scale,
                           weights=self.weights if weights is None else weights, decay=decay,
                           out=torch.full(self.weights.shape, -3.0, device="cuda") if out is None else out, window=self.window, sinks=self.sinks)

    def check(self, got):
        off = (got.double() - self.want).abs()
        assert bool((off <= self.limit).all()), f"{int((off > self.limit).sum())} of {off.numel()}, {float((off / self.limit.clamp(min=1e-300)).max())}"


def ragged(total, parts, seed):
    g = torch.Generator().manual_seed(seed)
    share = torch.rand(parts, generator=g) + 0.05
    return [max(1, int(x)) for x in share / share.sum() * total]


# Units are 128 tokens of a head for many rows to a head (a unit to one or, from 1024 rows (heads of 256: 512), two
# blocks), 32 to a warp for few, 256 to a block for heads of more queries than that.  152 SMs: more than 64
# units to a block or pair are 9728 and 4864; a warp's second tile begins at 1824 to 3648.
CASES = [
    # name, tokens in all, requests, queries of each (in turn), heads, kv heads, D, page, window, sinks
    ("tc 64", 160000, 9, [50, 1, 49], 16, 8, 64, 16, 0, 0),
    ("tc 128", 160000, 10, [70, 0, 3], 8, 8, 128, 64, 0, 0),
    ("tc 256", 160000, 8, [9, 17], 16, 4, 256, 32, 0, 0),
    ("tc 64 window", 60000, 5, [150], 8, 4, 64, 128, 2000, 70),
    ("tc 256 window", 40000, 4, [60, 33], 8, 8, 256, 16, 777, 0),
    ("pair 64", 90000, 7, [513, 40, 1], 16, 8, 64, 64, 0, 0),
    ("pair 128", 90000, 6, [300, 1], 32, 8, 128, 32, 0, 0),
    ("pair 256", 80000, 5, [90, 128, 7], 48, 8, 256, 64, 0, 0),
    ("pair 64 window", 30000, 3, [1100], 4, 4, 64, 16, 900, 5),
    ("few 64, 1 group of rows", 200000, 11, [1], 32, 8, 64, 16, 0, 0),
    ("few 64, 2", 200000, 11, [4, 0, 3], 32, 8, 64, 32, 0, 0),
    ("few 64, 3", 160000, 9, [6, 1], 32, 8, 64, 16, 0, 0),
    ("few 64, 4, window", 160000, 9, [8, 5], 32, 8, 64, 64, 3000, 40),
    ("few 64, 12", 120000, 7, [24, 1], 32, 8, 64, 16, 0, 0),
    ("few 128, 1", 200000, 13, [1], 32, 8, 128, 16, 0, 0),
    ("few 128, 1, window", 200000, 13, [2], 32, 8, 128, 64, 5000, 4),
    ("few 128, 2", 160000, 9, [4, 2], 32, 8, 128, 128, 0, 0),
    ("few 128, 3", 160000, 9, [5, 1], 32, 8, 128, 16, 0, 0),
    ("few 128, 8, window", 120000, 7, [16, 3], 32, 8, 128, 32, 400, 33),
    ("few 256, 1", 160000, 9, [1, 2], 32, 8, 256, 16, 0, 0),
    ("few 256, 2", 120000, 7, [4, 0, 1], 32, 8, 256, 64, 0, 0),
    ("few 256, 4", 100000, 6, [8, 7], 32, 8, 256, 32, 1500, 0),
    ("wide 64", 160000, 7, [2, 1], 260, 2, 64, 32, 0, 0),
    ("wide 128", 120000, 5, [1], 270, 2, 128, 16, 3000, 9),
    ("wide 256", 120000, 5, [3, 1], 130, 2, 256, 64, 0, 0),
]


def make(pn, name):
    _, total, parts, counts, heads, kv, D, page, window, sinks = next(c for c in CASES if c[0] == name)
    lens = ragged(total, parts, total + D)
    return Case(pn, lens, [min(counts[b % len(counts)], lens[b]) for b in range(parts)], heads, kv, D, page, window, sinks)


@pytest.mark.parametrize("name", [c[0] for c in CASES])
def test_many_units(pn, name):
    case = make(pn, name)
    got = case.call(pn)
    case.check(got)
    assert torch.equal(got, case.call(pn))
    mine = case.weights.clone()                              # in place
    case.call(pn, weights=mine, out=mine)
    assert torch.equal(mine, torch.where(got == -3, case.weights, got))


@pytest.mark.parametrize("name", ["tc 64", "tc 128", "tc 256 window", "pair 64", "pair 128", "pair 256"])
def test_waits_that_give_up(pn, name):
    """With limits that any wait may pass the call ends, an entry is right or NaN, none beside the tokens' is written, and the
    next call is right."""
    case = make(pn, name)
    right = case.call(pn)
    case.check(right)
    torch.cuda.synchronize()
    try:
        for ns in (1, 300, 1000, 2000, 4000, 8000, 16000, 50000):
            pn.set_wait_timeout_ns(ns)
            got = case.call(pn)
            torch.cuda.synchronize()
            there = got == right
            assert bool((there | torch.isnan(got)).all()), ns
            assert torch.equal(got[right == -3], right[right == -3])
    finally:
        pn.set_wait_timeout_ns(1_000_000_000)
    assert torch.equal(case.call(pn), right)


@pytest.mark.parametrize("heads,kv,D,counts", [(8, 2, 64, [1, 2]), (8, 2, 64, [5, 3]), (8, 2, 128, [1, 2]), (8, 2, 128, [3, 9]), (8, 2, 256, [2, 1]),
                                               (8, 2, 256, [6, 4]), (4, 2, 64, [90, 60]), (4, 2, 128, [70, 3]), (4, 2, 256, [60, 33]), (8, 2, 64, [300, 9]),
                                               (8, 2, 128, [290, 5]), (8, 2, 256, [140, 130]), (130, 1, 64, [2, 1]), (132, 1, 128, [1, 2]), (70, 1, 256, [2, 1])])
def test_no_bit_of_a_score_is_lost(pn, heads, kv, D, counts):
    """Two of each group's products are 2^15 times a code and cancel; what is left of the score are the others, which 20 bits
    beside them hold: products of whole numbers, as sums of 24 bits, keep them (of subnormals, which lie some 11 bits
    below their exponent, they would not)."""
    case = Case(pn, [500, 333], counts, heads, kv, D, 32, cancel=True)
    case.check(case.call(pn))
