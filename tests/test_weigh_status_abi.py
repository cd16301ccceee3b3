"""Argument checks of pn_kv_weigh_ex's workspace, without a GPU: every call here returns before the device is touched."""
from __future__ import annotations

import pytest

from test_step_operators_abi import PN_EALIGN, PN_EINVAL, PN_OK, WEIGH, at, lib  # noqa: F401

EX = {**{k: v for k, v in WEIGH.items() if k != "stream"}, "workspace": at(9), "workspace_bytes": 256, "stream": None}


@pytest.mark.parametrize("status,changes", [
    (PN_EINVAL, [dict(workspace_bytes=255), dict(workspace_bytes=0), dict(workspace=at(7)), dict(workspace=at(0)), dict(workspace=at(5)),
                 dict(workspace=at(6)), dict(workspace=at(1) + 256), dict(workspace=None, workspace_bytes=0, scale=float("nan")), dict(decay=2.0),
                 dict(out=None), dict(out=at(9) + 128)]),
    (PN_EALIGN, [dict(workspace=at(9) + 128), dict(workspace=at(9) + 4), dict(q=at(0) + 8)]),
    (PN_OK, [dict(tokens=0), dict(tokens=0, workspace=None, workspace_bytes=0)]),
])
def test_arguments(lib, status, changes):  # noqa: F811
    for change in changes:
        args = {**EX, **change}
        assert list(args) == list(EX)
        assert lib.pn_kv_weigh_ex(*args.values()) == status, change


def test_wrapper_looks_at_the_workspace(lib):  # noqa: F811
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    from bit_weight_only_pn_gb300 import pn

    class Other:
        def __init__(self, buffer):
            self.buffer = buffer

    def make(shape, dtype, device="cuda:0"):
        with FakeTensorMode():
            return torch.empty(shape, dtype=dtype, device=device)

    i32, f32, f16, u8 = torch.int32, torch.float32, torch.float16, torch.uint8
    args = [make((3, 4, 64), f16), make((4, 2, 1, 17 * 64), u8), make((2, 3), i32), make((2,), i32), make((3,), i32), 2, make((3, 4), f32), 0.1]
    out = make((4, 2, 16), f32)
    with pytest.raises(ValueError, match="must be on the device of"):
        pn.kv_weigh(*args, out=out, workspace=Other(make((512,), u8, "cuda:1")))
    with pytest.raises(TypeError):
        pn.kv_weigh(*args, out=out, workspace=Other(make((512,), f32)))
    with pytest.raises(TypeError):
        pn.kv_weigh(*args, out=out, workspace=Other(torch.zeros(512, dtype=u8)))
