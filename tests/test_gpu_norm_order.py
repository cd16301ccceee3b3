"""pn_norm's contract that a row's sums are made in one order whatever other rows there are: the same bits in calls of one
row, of as many as the GPU has SMs, and of more (where other splits of a row over threads are faster)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


@pytest.mark.parametrize("hidden", [1, 100, 1000, 1024, 1025, 1028, 2048, 4096, 4100, 5003, 5120, 6144, 6148, 8191, 8192, 8196, 10241, 12288, 16384,
                                    16385, 16388, 20479, 20480, 20484, 32764, 32767, 32768])
@pytest.mark.parametrize("post,pre,y_type,r_type", [(1, 1, torch.float32, torch.float32), (2, 2, torch.float16, torch.float16), (0, 2, torch.float16, torch.float32),
                                                    (1, 0, torch.float32, torch.float16)])
def test_rows_by_themselves(pn, hidden, post, pre, y_type, r_type):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(hidden)
    rows = 2 * sms + 3
    y = (torch.randn(rows, hidden, generator=g, device="cuda") * 2 + 3).to(y_type)
    r = (torch.randn(rows, hidden, generator=g, device="cuda") * 5).to(r_type)
    gate = torch.randn(rows, hidden, generator=g, device="cuda")
    weight, bias = (torch.randn(2, hidden, generator=g, device="cuda") for _ in range(2))

    def call(at):
        return pn.norm(y[at], r[at], gate[at], 0.37, post, weight[0] if post else None, bias[0] if post else None, pre, weight[1] if pre else None,
                       bias[1] if pre else None, 1e-5)

    whole = call(slice(None))
    for at in (slice(0, 1), slice(7, 8), slice(0, sms), slice(3, sms + 3), slice(0, sms + 1), slice(rows - 2, rows)):
        for got, want in zip(call(at), whole):
            assert torch.equal(got, want[at]), (at, int((got != want[at]).sum()))
