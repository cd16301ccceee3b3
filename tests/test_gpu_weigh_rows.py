"""pn_kv_weigh's rows that give nothing: lse of an infinity, whatever their queries hold."""
from __future__ import annotations

import math

import pytest
import torch

from test_gpu_weigh_units import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


# few rows to a head in registers, in shared memory; many, in one block and two; more heads than the kernel for many rows takes
FORMS = [(8, 2, 64, [1, 2]), (8, 2, 64, [5, 3]), (8, 2, 128, [1, 2]), (8, 2, 128, [3, 9]), (8, 2, 256, [2, 1]), (8, 2, 256, [6, 4]), (4, 2, 64, [90, 60]),
         (4, 2, 128, [70, 3]), (4, 2, 256, [60, 33]), (8, 2, 64, [300, 9]), (8, 2, 128, [290, 5]), (8, 2, 256, [140, 130]), (130, 1, 64, [2, 1]),
         (132, 1, 128, [1, 2]), (70, 1, 256, [2, 1])]


@pytest.mark.parametrize("heads,kv,D,counts", FORMS)
@pytest.mark.parametrize("window", [0, 100])
def test_rows_that_give_nothing(pn, heads, kv, D, counts, window):
    case = Case(pn, [777, 400], counts, heads, kv, D, 16, window, 3)
    g = torch.Generator(device="cuda").manual_seed(D)
    off = torch.rand(case.lse.shape, generator=g, device="cuda") < 0.3
    off[0, :2] = off[-1, -1] = True                          # (of the last row padding may be made)
    lse = case.lse.clone()
    case.lse[off] = -math.inf
    want = case.call(pn)
    assert not torch.isnan(want).any()
    for value in (math.nan, math.inf, -math.inf):
        case.q[off] = value
        assert torch.equal(case.call(pn), want), value
    case.lse[off] = math.inf
    assert torch.equal(case.call(pn), want)
    # and they give nothing at all: what is left are the other rows'
    case.lse[off] = lse[off]
    case.q[off] = 0
    both = case.call(pn, decay=0.0)
    case.lse[~off] = -math.inf
    theirs = case.call(pn, decay=0.0)
    case.lse = torch.where(off, -math.inf, lse)
    rest = case.call(pn, decay=0.0)
    written = both != -3
    assert torch.all((both - theirs - rest).abs()[written] <= 2.0 ** -17 * both[written])
