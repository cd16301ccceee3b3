"""pn_kv_weigh tells of a wait that gave up in a workspace's status word."""
from __future__ import annotations

import pytest
import torch

from test_gpu_weigh_units import Case

pytestmark = pytest.mark.gpu
PN_ETIMEOUT = 5


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


def call(pn, case, workspace):
    return pn.kv_weigh(case.q, case.cache, case.table, case.device_lens, case.starts, case.most, case.lse, case.scale, weights=case.weights, decay=0.9,
                       out=torch.full(case.weights.shape, -3.0, device="cuda"), workspace=workspace)


@pytest.mark.parametrize("make", ["attention", "gemv"])
@pytest.mark.parametrize("heads,kv,D,counts", [(4, 2, 64, [100, 60]), (4, 2, 128, [70, 3]), (4, 2, 256, [60, 33]), (8, 2, 128, [290, 5])])
def test_status(pn, make, heads, kv, D, counts):
    case = Case(pn, [900, 500], counts, heads, kv, D, 16)
    workspace = pn.AttentionWorkspace() if make == "attention" else pn.Workspace(1024)
    got = call(pn, case, workspace)
    case.check(got)
    assert workspace.status() == 0
    pn.set_wait_timeout_ns(5_000_000)
    pn.set_test_stall(True)
    try:
        lost = call(pn, case, workspace)
        torch.cuda.synchronize()
    finally:
        pn.set_test_stall(False)
        pn.set_wait_timeout_ns(1_000_000_000)
    assert torch.isnan(lost).any() and not torch.isnan(got).any()
    assert workspace.status() == PN_ETIMEOUT
    assert workspace.status() == 0 and not workspace.buffer.any()
    assert torch.equal(call(pn, case, workspace), got) and workspace.status() == 0
    if make == "attention":                                  # which works on with it
        args = (case.q, case.cache, case.table, case.device_lens, case.starts, case.most, case.scale)
        assert torch.equal(pn.attention(*args, workspace=workspace), pn.attention(*args))


def test_limits_that_any_wait_may_pass(pn):
    """Wherever a weight is NaN, the status word says so."""
    case = Case(pn, [9000, 5000, 700], [290, 5, 100], 8, 2, 128, 16)
    workspace = pn.Workspace(1024)
    right = call(pn, case, workspace)
    case.check(right)
    try:
        for ns in (1, 500, 1000, 2000, 3000, 5000, 10000, 30000):
            pn.set_wait_timeout_ns(ns)
            got = call(pn, case, workspace)
            status = workspace.status()
            assert bool(((got == right) | torch.isnan(got)).all())
            assert status in (0, PN_ETIMEOUT) and (status or not torch.isnan(got).any()), ns
    finally:
        pn.set_wait_timeout_ns(1_000_000_000)
    assert torch.equal(call(pn, case, workspace), right) and workspace.status() == 0


def test_kernels_without_waits(pn):
    case = Case(pn, [900, 500], [2, 1], 8, 2, 128, 16)
    workspace = pn.Workspace(64)
    case.check(call(pn, case, workspace))
    assert workspace.status() == 0
