"""Argument checks of the serving-step calls of the C ABI, and their restatements
against one another.  Without a GPU: every call here returns before the device
is touched, and addresses are never read.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import serving_ref as ref

PN_OK, PN_EINVAL, PN_EALIGN = 0, 1, 2
NAN = float("nan")


def at(i):
    return 0x100000000 * (i + 1)                      # addresses 4 GiB apart


@pytest.fixture(scope="module")
def lib():
    from bit_weight_only_pn_gb300 import build, pn
    build.build()
    return pn.lib()


def test_cache_bytes(lib):
    f = lib.pn_kv_cache_bytes
    for pages, page, heads, D in ((1, 16, 1, 64), (7, 64, 8, 128), (100000, 1024, 8, 256)):
        assert f(pages, page, heads, D) == pages * heads * page // 16 * 17 * D
    for bad in ((0, 16, 1, 64), (-1, 16, 1, 64), (1, 8, 1, 64), (1, 24, 1, 64), (1, 2048, 1, 64), (1, 16, 0, 64), (1, 16, 1, 96), (1, 16, 1, 512)):
        assert f(*bad) == 0


PLAN = dict(lens=at(0), add=at(1), held=at(2), batch=4, table=at(3), table_stride=8, max_pages=8, free_pages=at(4), pages=64, ring=at(5),
            page_size=16, capacity=32, slots=at(6), positions=at(7), requests=at(8), starts=at(9), lens_out=at(10), held_out=at(11),
            ring_out=at(12), refused=at(13), stream=None)
APPEND = dict(q=at(0), q_stride=512, k=at(1), k_stride=128, v=at(2), v_stride=128, dtype=0, tokens=3, heads=8, q_weight=at(3), k_weight=at(4),
              eps=1e-6, cos=at(5), sin=at(6), table_rows=100, rotary=64, interleaved=0, positions=at(7), slots=at(8), cache=at(9), pages=4,
              page_size=16, kv_heads=2, head_dim=64, q_out=at(10), stream=None)
READ = dict(cache=at(0), pages=4, page_size=16, kv_heads=2, head_dim=64, slots=at(1), tokens=3, k=at(2), v=at(3), stream=None)
ATTENTION = dict(q=at(0), q_stride=512, tokens=3, heads=8, cache=at(1), pages=4, page_size=16, kv_heads=2, head_dim=64, table=at(2),
                 table_stride=4, max_pages=4, lens=at(3), starts=at(4), batch=2, max_queries=2, scale=0.1, window=0, sinks=0, out=at(5),
                 lse=at(6), workspace=at(7), workspace_bytes=1 << 30, stream=None)
VERIFY = dict(tokens=at(0), target=at(1), target_stride=100, draft=at(2), draft_stride=100, uniforms=at(3), counts=at(4), batch=2, drafts=3,
              vocab=100, accepted=at(5), out=at(6), stream=None)

REFUSED = [
    ("pn_kv_plan", PLAN, PN_EINVAL, [dict(batch=0), dict(batch=16385), dict(max_pages=0), dict(table_stride=7), dict(pages=0),
                                     dict(pages=1 << 31), dict(page_size=24), dict(page_size=8), dict(capacity=-1), dict(capacity=1 << 31),
                                     dict(max_pages=1 << 27, table_stride=1 << 27), dict(lens=None), dict(slots=None), dict(refused=None),
                                     dict(lens_out=at(0)), dict(table=at(0)), dict(ring_out=at(5)), dict(slots=at(7)), dict(starts=at(9), held_out=at(9) + 16)]),
    ("pn_kv_plan", PLAN, PN_EALIGN, [dict(lens=at(0) + 2), dict(ring=at(5) + 4), dict(slots=at(6) + 4), dict(refused=at(13) + 1)]),
    ("pn_kv_append", APPEND, PN_EINVAL, [dict(head_dim=96), dict(page_size=20), dict(kv_heads=0), dict(pages=0), dict(dtype=2), dict(tokens=-1),
                                         dict(heads=-1), dict(heads=65537), dict(rotary=63), dict(rotary=66), dict(rotary=-2), dict(eps=-1.0),
                                         dict(eps=NAN), dict(q=None), dict(k=None), dict(slots=None), dict(cos=None), dict(positions=None),
                                         dict(q_stride=511), dict(k_stride=127), dict(v_stride=0), dict(q_out=at(0)), dict(cache=at(1))]),
    ("pn_kv_append", APPEND, PN_EALIGN, [dict(q=at(0) + 2), dict(k_weight=at(4) + 1), dict(cache=at(9) + 8), dict(q_out=at(10) + 8),
                                         dict(slots=at(8) + 4), dict(positions=at(7) + 2)]),
    ("pn_kv_append", APPEND, PN_OK, [dict(tokens=0), dict(tokens=0, q=None, k=None, v=None, cache=None)]),
    ("pn_kv_read", READ, PN_EINVAL, [dict(head_dim=65), dict(tokens=-1), dict(cache=None), dict(k=None), dict(k=at(3)), dict(v=at(0))]),
    ("pn_kv_read", READ, PN_EALIGN, [dict(k=at(2) + 4), dict(slots=at(1) + 4)]),
    ("pn_kv_read", READ, PN_OK, [dict(tokens=0)]),
    ("pn_attention", ATTENTION, PN_EINVAL, [dict(heads=7), dict(heads=0), dict(batch=0), dict(batch=16385), dict(max_queries=0), dict(max_pages=0),
                                            dict(table_stride=3), dict(window=-1), dict(sinks=-1), dict(scale=NAN), dict(scale=math.inf),
                                            dict(q_stride=504), dict(tokens=-1), dict(tokens=1 << 31), dict(max_queries=1 << 30),
                                            dict(max_pages=1 << 28, table_stride=1 << 28), dict(out=at(0)), dict(out=at(1)), dict(q=None),
                                            dict(workspace=None), dict(head_dim=32)]),
    ("pn_attention", ATTENTION, PN_EALIGN, [dict(q=at(0) + 8), dict(q_stride=513), dict(workspace=at(7) + 128), dict(lse=at(6) + 2),
                                            dict(cache=at(1) + 8), dict(table=at(2) + 2)]),
    ("pn_attention", ATTENTION, PN_OK, [dict(tokens=0)]),
    ("pn_verify", VERIFY, PN_EINVAL, [dict(batch=-1), dict(drafts=32), dict(drafts=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1, target_stride=1 << 21),
                                      dict(target_stride=99), dict(draft_stride=99), dict(tokens=None), dict(uniforms=None), dict(out=None),
                                      dict(out=at(0)), dict(accepted=at(6))]),
    ("pn_verify", VERIFY, PN_EALIGN, [dict(target=at(1) + 2), dict(counts=at(4) + 1), dict(out=at(6) + 3)]),
    ("pn_verify", VERIFY, PN_OK, [dict(batch=0)]),
]


@pytest.mark.parametrize("name,good,status,changes", REFUSED, ids=[f"{r[0]}-{r[2]}" for r in REFUSED])
def test_arguments(lib, name, good, status, changes):
    for change in changes:
        args = {**good, **change}
        assert list(args) == list(good)
        assert getattr(lib, name)(*args.values()) == status, change


@pytest.mark.parametrize("D", [64, 128, 256])
def test_record_layout(D):
    """Every code and scale of a record has a place of its own, and what is written there reads back."""
    rng = np.random.default_rng(D)
    x = rng.standard_normal((16, 1, D)).astype(np.float32)
    n, d = ref.quantise(x)
    cache = np.zeros((1, 1, 1, 17 * D), np.uint8)
    ref.write_tokens(cache, range(16), n, d, n, d)
    assert np.abs(ref.dequantise(n, d) - x).max() <= np.abs(x).max() / 8      # half a step of at most max / 4
    other = np.full_like(cache, 0xFF)
    ref.write_tokens(other, range(16), n, d, n, d)
    assert np.array_equal(cache, other)                                       # no byte of a full record is left out


def test_attention_reference_against_differences():
    """The restatement's log-sum-exp has the outputs' weights as its gradient: values = keys' gradient of lse."""
    rng = np.random.default_rng(0)
    L, D, scale = 9, 64, 0.2
    q = rng.standard_normal((1, 1, D))
    k = rng.standard_normal((L, 1, D)).astype(np.float32)
    v = k.copy()
    out, lse, *_ = ref.attention(q, k, v, scale, 0, 0)
    step = 1e-5
    for i in (0, 5, 63):                                                      # d lse / d q = scale * sum p k = scale * out
        moved = q.copy()
        moved[0, 0, i] += step
        back = q.copy()
        back[0, 0, i] -= step
        slope = (ref.attention(moved, k, v, scale, 0, 0)[1] - ref.attention(back, k, v, scale, 0, 0)[1]) / (2 * step)
        assert abs(slope[0, 0] - scale * out[0, 0, i]) < 1e-8


def test_wrappers_refuse_cpu_tensors():
    import torch
    from bit_weight_only_pn_gb300 import pn
    cpu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        pn.kv_plan(cpu, cpu, cpu, torch.zeros(2, 2, dtype=torch.int32), cpu, torch.zeros(2, dtype=torch.int64), 16, 2)


def test_attention_work_past_32_bits(lib):
    """Refused on the host: row groups as max_queries allows for, and units by the queries there are."""
    base = {**ATTENTION, "kv_heads": 8, "q_stride": 512, "batch": 16384}
    for change in (dict(max_queries=1 << 18), dict(max_queries=1 << 17, head_dim=256, q_stride=2048),   # 2^14 x 8 x 2^14 row groups
                   dict(batch=4, tokens=1 << 20, max_queries=1 << 20, max_pages=1 << 26, table_stride=1 << 26),
                   dict(tokens=1 << 20, max_queries=64, max_pages=1 << 18, table_stride=1 << 18, table=at(100))):   # 2^14 x 8 x 2^16
        args = {**base, **change}
        assert list(args) == list(ATTENTION)
        assert lib.pn_attention(*args.values()) == 3, change


SHARED = [
    ("pn_kv_append", APPEND, [dict(q_out=at(9) + 64), dict(q_out=at(3)), dict(q_out=at(4)), dict(q_out=at(5)), dict(q_out=at(6)), dict(q_out=at(7)),
                              dict(q_out=at(8)), dict(cache=at(8)), dict(cache=at(5)), dict(cache=at(3)), dict(q_out=at(1) + 256), dict(cache=at(2))]),
    ("pn_kv_read", READ, [dict(k=at(1)), dict(v=at(1)), dict(v=at(2) + 512)]),
    ("pn_attention", ATTENTION, [dict(out=at(2)), dict(out=at(3)), dict(out=at(4)), dict(out=at(7) + 4096), dict(lse=at(0)), dict(lse=at(1) + 4),
                                 dict(lse=at(2)), dict(lse=at(3)), dict(lse=at(4) + 8), dict(lse=at(5) + 32), dict(lse=at(7)), dict(workspace=at(0)),
                                 dict(workspace=at(3)), dict(workspace=at(1))]),
    ("pn_verify", VERIFY, [dict(accepted=at(4)), dict(accepted=at(0)), dict(accepted=at(3) + 4), dict(accepted=at(1)), dict(accepted=at(2) + 2396),
                           dict(out=at(1) + 3196), dict(out=at(2)), dict(out=at(3)), dict(out=at(4) + 4), dict(counts=at(5) + 4)]),
]


@pytest.mark.parametrize("name,good,changes", SHARED, ids=[r[0] for r in SHARED])
def test_outputs_share_no_memory(lib, name, good, changes):
    for change in changes:
        assert getattr(lib, name)(*{**good, **change}.values()) == PN_EINVAL, change


def test_wrappers_refuse_tensors_of_two_devices(lib):
    """Tensors without memory that stand for two GPUs': every argument of every call is looked at before anything else is done."""
    import types

    import torch
    from torch._subclasses.fake_tensor import FakeTensorMode
    from bit_weight_only_pn_gb300 import pn
    i32, i64, f32, f16, u8 = torch.int32, torch.int64, torch.float32, torch.float16, torch.uint8
    mode = FakeTensorMode()

    def make(shape, dtype, device):
        with mode:
            return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")

    plan_out = [((4,), i64), ((4,), i32), ((4,), i32), ((3,), i32), ((2,), i32), ((2,), i32), ((2,), i64), ((1,), i32)]
    plan_args = [((2,), i32)] * 3 + [((2, 3), i32), ((9,), i32), ((2,), i64)]
    cache, token = ((4, 2, 1, 17 * 64), u8), ((3, 2, 64), f32)
    calls = {
        "plan": (plan_args, lambda t: pn.kv_plan(*t, 16, 4)),
        "plan into": (plan_args + plan_out, lambda t: pn.kv_plan(*t[:6], 16, 4, out=pn.KvPlan(*t[6:]))),
        "append": ([token, token, token, cache, ((3,), i64), ((3,), i32), ((5, 32), f32), ((5, 32), f32), ((64,), f32), ((64,), f32), ((3, 2, 64), f16)],
                   lambda t: pn.kv_append(*t[:10], q_out=t[10])),
        "read": ([cache, ((3,), i64), token, token], lambda t: pn.kv_read(t[0], t[1], out=(t[2], t[3]))),
        "attention": ([((3, 4, 64), f16), cache, ((2, 3), i32), ((2,), i32), ((3,), i32), ((3, 4, 64), f16), ((3, 4), f32), ((1 << 20,), u8)],
                      lambda t: pn.attention(*t[:5], 2, 0.1, out=t[5], lse=t[6], workspace=types.SimpleNamespace(buffer=t[7]))),
        "verify": ([((2, 3), i32), ((2, 4, 10), f32), ((2, 3, 10), f32), ((2, 4), f32), ((2,), i32), ((2,), i32), ((2, 4), i32)],
                   lambda t: pn.verify(*t[:4], counts=t[4], accepted=t[5], out=t[6])),
    }
    for name, (shapes, call) in calls.items():
        for other in range(len(shapes)):
            with pytest.raises(ValueError, match="must be on the device of"):
                call([make(s, d, int(i == other)) for i, (s, d) in enumerate(shapes)])


def test_cache_bytes_past_63_bits(lib):
    """Shapes whose bytes do not fit are refused, not taken modulo 2^64."""
    f, most = lib.pn_kv_cache_bytes, (1 << 31) - 1
    per_page = 65536 * 64 * 17 * 256
    pages = ((1 << 63) - 1) // per_page
    assert f(pages, 1024, 65536, 256) == pages * per_page
    for shape in ((pages + 1, 1024, 65536, 256), (most, 1024, 65536, 256), (most, 1024, 65536, 64), (1 << 30, 1024, 65536, 128)):
        exact = shape[0] * shape[2] * (shape[1] // 16) * 17 * shape[3]
        assert f(*shape) == (exact if exact < 1 << 63 else 0)
        if exact >= 1 << 63:
            change = dict(zip(("pages", "page_size", "kv_heads", "head_dim"), shape))
            for name, good in (("pn_kv_append", APPEND), ("pn_kv_read", READ), ("pn_attention", ATTENTION)):
                assert getattr(lib, name)(*{**good, **change}.values()) == PN_EINVAL
