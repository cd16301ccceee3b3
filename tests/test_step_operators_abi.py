"""Argument checks of pn_logprobs, pn_norm, pn_kv_weigh and pn_kv_evict.  Without a
GPU: every call here returns before the device is touched, and addresses are never read.
"""
from __future__ import annotations

import math

import pytest

PN_OK, PN_EINVAL, PN_EALIGN = 0, 1, 2
NAN = float("nan")
MOST = (1 << 31) - 1


def at(i):
    return 0x100000000 * (i + 1)                      # addresses 4 GiB apart


@pytest.fixture(scope="module")
def lib():
    from bit_weight_only_pn_gb300 import build, pn
    build.build()
    return pn.lib()


LOGPROBS = dict(logits=at(0), stride=100, dtype=0, rows=3, vocab=100, scale=1.0, tokens=at(1), count=2, logprobs=at(2), entropy=at(3), top=5,
                top_tokens=at(4), top_logprobs=at(5), stream=None)
NORM = dict(y=at(0), y_stride=64, y_dtype=0, residual=at(1), residual_stride=64, residual_dtype=0, gate=at(2), gate_stride=64, scale=1.0, tokens=3,
            hidden=64, post=1, post_weight=at(3), post_bias=at(4), pre=2, pre_weight=at(5), pre_bias=at(6), eps=1e-6, residual_out=at(7),
            out_stride=64, x=at(8), stream=None)
WEIGH = dict(q=at(0), q_stride=512, tokens=3, heads=8, cache=at(1), pages=4, page_size=16, kv_heads=2, head_dim=64, table=at(2), table_stride=4,
             max_pages=4, lens=at(3), starts=at(4), batch=2, max_queries=2, lse=at(5), scale=0.1, window=0, sinks=0, weights=at(6), decay=1.0,
             out=at(7), stream=None)
EVICT = dict(cache=at(0), pages=4, page_size=16, kv_heads=2, head_dim=64, weights=at(1), table=at(2), table_stride=4, max_pages=4, lens=at(3),
             held=at(4), batch=2, limit=40, budget=20, sinks=2, recent=8, free_pages=at(5), ring_pages=4, ring=at(6), table_out=at(7), out_stride=4,
             lens_out=at(8), held_out=at(9), ring_out=at(10), kept=at(11), refused=at(12), stream=None)

REFUSED = [
    ("pn_logprobs", LOGPROBS, PN_EINVAL, [dict(dtype=2), dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 20) + 1, stride=1 << 21),
                                          dict(stride=99), dict(stride=1 << 40), dict(count=-1), dict(top=-1), dict(top=33), dict(scale=0.0),
                                          dict(scale=-1.0), dict(scale=NAN), dict(scale=math.inf), dict(scale=1e-30), dict(logits=None),
                                          dict(tokens=None), dict(logprobs=None), dict(top_tokens=None), dict(top_logprobs=None),
                                          dict(logprobs=at(0)), dict(entropy=at(1)), dict(top_tokens=at(0) + 1196), dict(top_logprobs=at(4)),
                                          dict(entropy=at(2) + 20)]),
    ("pn_logprobs", LOGPROBS, PN_EALIGN, [dict(logits=at(0) + 2), dict(logits=at(0) + 1, dtype=1), dict(tokens=at(1) + 2), dict(logprobs=at(2) + 1),
                                          dict(entropy=at(3) + 2), dict(top_tokens=at(4) + 1), dict(top_logprobs=at(5) + 2)]),
    ("pn_logprobs", LOGPROBS, PN_OK, [dict(rows=0), dict(rows=0, logits=None, tokens=None)]),
    ("pn_norm", NORM, PN_EINVAL, [dict(y_dtype=2), dict(residual_dtype=-1), dict(post=3), dict(pre=-1), dict(tokens=-1), dict(tokens=1 << 31),
                                  dict(hidden=0), dict(hidden=32769, y_stride=1 << 16, residual_stride=1 << 16, out_stride=1 << 16, gate_stride=0),
                                  dict(eps=-1.0), dict(eps=NAN), dict(scale=NAN), dict(scale=math.inf), dict(post=0), dict(pre=0),
                                  dict(post=0, post_weight=None), dict(y=None), dict(y=None, gate=None), dict(x=None), dict(y=None, residual=None, gate=None, post=0, post_weight=None, post_bias=None),
                                  dict(residual_out=None, x=None, pre=0, pre_weight=None, pre_bias=None), dict(y_stride=63), dict(residual_stride=63),
                                  dict(gate_stride=63), dict(gate_stride=-64), dict(out_stride=63), dict(y_stride=1 << 40), dict(residual_out=at(0)),
                                  dict(residual_out=at(1), out_stride=65), dict(residual_out=at(1) + 4), dict(x=at(1)), dict(x=at(7) + 4),
                                  dict(x=at(2)), dict(x=at(5)), dict(residual_out=at(3))]),
    ("pn_norm", NORM, PN_EALIGN, [dict(y=at(0) + 2), dict(y=at(0) + 1, y_dtype=1), dict(residual=at(1) + 2), dict(residual_out=at(7) + 2), dict(gate=at(2) + 2),
                                  dict(post_weight=at(3) + 2), dict(pre_bias=at(6) + 1), dict(x=at(8) + 1)]),
    ("pn_norm", NORM, PN_OK, [dict(tokens=0), dict(tokens=0, y=at(0), residual=None)]),
    ("pn_kv_weigh", WEIGH, PN_EINVAL, [dict(head_dim=96), dict(page_size=24), dict(heads=7), dict(heads=0), dict(batch=0), dict(batch=16385),
                                       dict(max_queries=0), dict(max_pages=0), dict(table_stride=3), dict(window=-1), dict(sinks=-1), dict(scale=NAN),
                                       dict(decay=-0.1), dict(decay=1.5), dict(decay=NAN), dict(q_stride=504), dict(tokens=-1), dict(tokens=1 << 31),
                                       dict(max_queries=1 << 30), dict(max_pages=1 << 27, table_stride=1 << 27), dict(q=None), dict(lse=None),
                                       dict(out=None), dict(cache=None), dict(out=at(0)), dict(out=at(1) + 4), dict(out=at(2)), dict(out=at(3)),
                                       dict(out=at(4)), dict(out=at(5)), dict(out=at(6) + 64)]),
    ("pn_kv_weigh", WEIGH, PN_EALIGN, [dict(q=at(0) + 8), dict(q_stride=513), dict(cache=at(1) + 8), dict(table=at(2) + 2), dict(lse=at(5) + 1),
                                       dict(weights=at(6) + 2), dict(out=at(7) + 2)]),
    ("pn_kv_weigh", WEIGH, PN_OK, [dict(tokens=0)]),
    ("pn_kv_evict", EVICT, PN_EINVAL, [dict(head_dim=32), dict(pages=0), dict(batch=0), dict(batch=16385), dict(max_pages=0), dict(table_stride=3),
                                       dict(out_stride=3), dict(ring_pages=0), dict(ring_pages=1 << 31), dict(budget=0), dict(budget=41),
                                       dict(budget=(1 << 23) + 1, limit=MOST), dict(sinks=-1), dict(recent=-1), dict(sinks=13), dict(sinks=MOST, recent=MOST),
                                       dict(max_pages=1 << 27, table_stride=1 << 27, out_stride=1 << 27), dict(cache=None), dict(weights=None),
                                       dict(kept=None), dict(refused=None), dict(ring=None), dict(table_out=at(2)), dict(lens_out=at(3)),
                                       dict(held_out=at(4)), dict(ring_out=at(6)), dict(kept=at(0)), dict(kept=at(1)), dict(weights=at(0)),
                                       dict(free_pages=at(2)), dict(table_out=at(5)), dict(refused=at(11) + 4)]),
    ("pn_kv_evict", EVICT, PN_EALIGN, [dict(cache=at(0) + 8), dict(weights=at(1) + 2), dict(ring=at(6) + 4), dict(ring_out=at(10) + 4), dict(kept=at(11) + 2),
                                       dict(lens=at(3) + 1)]),
]


@pytest.mark.parametrize("name,good,status,changes", REFUSED, ids=[f"{r[0]}-{r[2]}" for r in REFUSED])
def test_arguments(lib, name, good, status, changes):
    for change in changes:
        args = {**good, **change}
        assert list(args) == list(good)
        assert getattr(lib, name)(*args.values()) == status, change


def test_wrappers_refuse_what_is_no_cuda_tensor(lib):
    import torch
    from bit_weight_only_pn_gb300 import pn
    x = torch.zeros(2, 64)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        pn.logprobs(x)
    with pytest.raises(TypeError):
        pn.norm(x)
    with pytest.raises(TypeError):
        pn.norm(None, None)
    with pytest.raises(TypeError):
        pn.kv_weigh(x, x, i32, i32, i32, 1, x, 1.0, out=x)
    with pytest.raises(TypeError):
        pn.kv_evict(x, x, i32, i32, i32, i32, i32, 4, 2)


def test_wrappers_refuse_tensors_of_two_devices(lib):
    """Tensors without memory that stand for two GPUs': every argument of every call is looked at before anything else is done."""
    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    from bit_weight_only_pn_gb300 import pn
    i32, i64, f32, f16, u8 = torch.int32, torch.int64, torch.float32, torch.float16, torch.uint8
    mode = FakeTensorMode()

    def make(shape, dtype, device):
        with mode:
            return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")

    cache, weights, row = ((4, 2, 1, 17 * 64), u8), ((4, 2, 16), f32), ((3, 64), f32)
    evict = [cache, weights, ((2, 3), i32), ((2,), i32), ((2,), i32), ((9,), i32), ((2,), i64)]
    evicted = [((2, 3), i32), ((2,), i32), ((2,), i32), ((2,), i64), ((2, 2, 5), i32), ((1,), i32)]
    calls = {
        "logprobs": ([row, ((3,), i32)], lambda t: pn.logprobs(*t)),
        "norm": ([row, row, ((64,), f32), ((64,), f32), ((64,), f32), ((64,), f32), ((64,), f32), row, ((3, 64), f16)],
                 lambda t: pn.norm(t[0], t[1], t[2], post=1, post_weight=t[3], post_bias=t[4], pre_weight=t[5], pre_bias=t[6], residual_out=t[7], x=t[8])),
        "weigh": ([((3, 4, 64), f16), cache, ((2, 3), i32), ((2,), i32), ((3,), i32), ((3, 4), f32), weights, weights],
                  lambda t: pn.kv_weigh(*t[:5], 2, t[5], 0.1, weights=t[6], out=t[7])),
        "evict": (evict, lambda t: pn.kv_evict(*t, 10, 5)),
        "evict into": (evict + evicted, lambda t: pn.kv_evict(*t[:7], 10, 5, out=pn.KvEviction(*t[7:]))),
    }
    for name, (shapes, call) in calls.items():
        for other in range(len(shapes)):
            with pytest.raises(ValueError, match="must be on the device of"):
                call([make(s, d, int(i == other)) for i, (s, d) in enumerate(shapes)])
