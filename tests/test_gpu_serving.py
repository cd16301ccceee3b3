"""The serving-step operators (pn_kv_plan, pn_kv_append, pn_kv_read, pn_attention,
pn_verify) against plain 64-bit and integer restatements.

Tolerances.  Plans, codes, cache bytes and verified tokens: equal.  Queries of
pn_kv_append: the documented fp32 arithmetic rounded to fp16, equal.

Attention.  With x_t the scores: fp32 accumulation of exact products, 64 to a
group, errs by at most 2^-19 of scale * sum |q| |k| (`reach`); the exponent's
argument and its reference are fp32 (2^-24 each of their size, taken four
times), ex2 and the fp32 sums add 2^-21 + L 2^-24 for L tokens.  So every
p_t, and their sum, carries a relative error of at most
  e = 2^-19 reach + 2^-22 (1.5 max(|x|, 10) + 14) + 2^-21 + L 2^-24,
where |x| <= reach.  p_t d_t is rounded once to fp16 (2^-11), small ones to
2^-25 against a largest of 2^13 at least (2^-38, times |n - 8| <= 8 and L
tokens); the output is rounded to fp16 (2^-11, or 2^-25 among subnormals):
  |out - exact| <= (2^-11 + 2 e) sum p |v| + L 2^-35 max|v| + 2^-11 |exact| + 2^-25
  |lse - exact| <= 2 e + 2^-22 |exact|
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# --------------------------------------------------------------------- plan --
PLANS = [
    # batch, page, longest, most new, free pages (None: plenty), capacity (None: all), finished share
    (1, 16, 0, 1, None, None, 0.0), (1, 64, 100, 0, None, None, 0.0), (3, 16, 40, 5, None, None, 0.3),
    (7, 32, 200, 70, 6, None, 0.2), (33, 16, 100, 9, 10, 60, 0.1), (300, 128, 4000, 200, 40, None, 0.1),
    (1024, 16, 64, 3, None, None, 0.5), (1500, 64, 500, 17, 300, 9000, 0.05), (5000, 16, 33, 2, 900, None, 0.1),
    (16384, 16, 40, 2, 3000, None, 0.3),
]


@pytest.mark.parametrize("batch,page,longest,new,free_pages,capacity,finished", PLANS)
def test_plan(pn, batch, page, longest, new, free_pages, capacity, finished):
    rng = np.random.default_rng(batch + page)
    lens = rng.integers(0, longest + 1, batch).astype(np.int32)
    add = rng.integers(0, new + 1, batch).astype(np.int32)
    add[rng.random(batch) < finished] = -1
    held = (-(-lens // page) + (rng.random(batch) < 0.3)).astype(np.int32)
    most = (longest + new) // page + 2
    if batch == 7:
        most -= 2                                   # some requests pass the table
        lens = np.minimum(lens, most * page)
        held = np.minimum(held, most)
    used = int(held.sum())
    spare = free_pages if free_pages is not None else batch * (new // page + 2)
    F = used + spare
    order = rng.permutation(F).astype(np.int32)
    wide = np.full((batch, most + 3), -7, np.int32)   # rows longer than the pages in use
    table = wide[:, :most]
    at = 0
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head = int(rng.integers(0, 3 * F))
    free = np.full(F, -5, np.int32)
    for i in range(spare):
        free[(head + i) % F] = order[used + i]
    ring = np.array([head, head + spare], np.int64)
    total = int(np.maximum(add, 0).sum())
    T = total + 5 if capacity is None else capacity
    d_wide, d_free = cuda(wide), cuda(free)
    got = pn.kv_plan(cuda(lens), cuda(add), cuda(held), d_wide[:, :most], d_free, cuda(ring), page, T)
    want = ref.plan(lens, add, held, table, free, ring, page, T)
    for name in got._fields:
        assert getattr(got, name).cpu().tolist() == want[name], name
    assert np.array_equal(d_wide.cpu().numpy(), wide)
    assert np.array_equal(d_free.cpu().numpy(), free)
    # again on the same inputs, into the same outputs
    again = pn.kv_plan(cuda(lens), cuda(add), cuda(held), d_wide[:, :most], d_free, cuda(ring), page, T, out=got)
    for name in got._fields:
        assert getattr(again, name).cpu().tolist() == want[name], name


def test_plan_state_goes_round(pn):
    """Requests come, grow, lose drafts and finish over many steps: no page is lost or lent twice."""
    rng = np.random.default_rng(5)
    B, page, most, F, T = 12, 16, 8, 60, 200
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(F, dtype=torch.int32, device="cuda")
    lens, held = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    ring = torch.tensor([0, F], device="cuda")
    for step in range(40):
        add = cuda(np.where(rng.random(B) < 0.15, -1, rng.integers(0, 17, B)).astype(np.int32))
        p = pn.kv_plan(lens, add, held, table, free, ring, page, T)
        lens, held, ring = p.lens, p.held, p.ring
        h, tab, fr = held.cpu().numpy(), table.cpu().numpy(), free.cpu().numpy()
        head, tail = ring.cpu().tolist()
        mine = [int(x) for b in range(B) for x in tab[b, :h[b]]]
        idle = [int(fr[i % F]) for i in range(head, tail)]
        assert sorted(mine + idle) == list(range(F)), step
        slots = [s for s in p.slots.cpu().tolist() if s >= 0]
        assert len(set(slots)) == len(slots)
        lens = torch.clamp(lens - cuda(rng.integers(0, 4, B).astype(np.int32)), min=0)   # drafts turned down


def test_plan_refusals(pn):
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, add, held = (torch.zeros(4, **i32) for _ in range(3))
    table, free, ring = torch.zeros(4, 3, **i32), torch.zeros(9, **i32), torch.tensor([0, 9], device="cuda")
    for page in (0, 8, 24, 2048):
        with pytest.raises(pn.PnError) as e:
            pn.kv_plan(lens, add, held, table, free, ring, page, 4)
        assert e.value.status == 1
    with pytest.raises(TypeError):
        pn.kv_plan(lens.long(), add, held, table, free, ring, 16, 4)
    with pytest.raises(ValueError):
        pn.kv_plan(lens, add[:3], held, table, free, ring, 16, 4)
    with pytest.raises(ValueError):
        pn.kv_plan(lens, add, held, table, free, ring, 16, -1)
    ok = pn.kv_plan(lens, add, held, table, free, ring, 16, 4)
    with pytest.raises(pn.PnError) as e:             # the state of a call may not be its output
        pn.kv_plan(ok.lens, add, ok.held, table, free, ok.ring, 16, 4, out=ok)
    assert e.value.status == 1
    assert pn.kv_plan(lens, add, held, table, free, ring, 16, 0).slots.numel() == 0


# ------------------------------------------------------------ append and read --
APPENDS = [
    # tokens, heads, kv heads, D, page, rotary, interleaved, norm, dtype, fused rows
    (1, 1, 1, 64, 16, 64, False, True, "f32", False), (1, 24, 4, 256, 16, 64, False, True, "f32", False),
    (2, 6, 2, 128, 32, 128, False, True, "f16", True), (5, 3, 3, 64, 16, 2, True, False, "f16", True),
    (17, 8, 1, 256, 64, 256, True, True, "f32", True), (33, 4, 2, 128, 16, 96, False, False, "f32", False),
    (40, 5, 5, 64, 128, 0, False, True, "f16", False), (130, 0, 2, 128, 64, 64, True, True, "f32", False),
    (300, 12, 2, 128, 16, 34, False, True, "f16", True),
]


def append_case(tokens, heads, kv, D, page, rotary, interleaved, norm, dtype, fused, seed=0):
    rng = np.random.default_rng(tokens * 7 + D + seed)
    np_t = np.float32 if dtype == "f32" else np.float16
    rows = (rng.standard_normal((tokens, (heads + 2 * kv) * D + 16)) * 2.0 ** rng.integers(-3, 4, (tokens, 1))).astype(np_t)
    rows[0, :] = 0                                    # a zero token: zero blocks
    if tokens > 1:
        rows[1, ::3] = np_t(1.5)                       # ties of the largest magnitude, both signs
        rows[1, 1::3] = np_t(-1.5)
        rows[1, 2::3] = np_t(0.25)
    d = cuda(rows)
    cut = [heads * D, kv * D, kv * D, 16]
    q, k, v, _ = d.split(cut, dim=1)
    parts = [x.unflatten(1, (-1, D)) if x.shape[1] else None for x in (q, k, v)]
    if not fused:
        parts = [None if x is None else x.contiguous() for x in parts]
    host = np.split(rows, np.cumsum(cut)[:-1], axis=1)[:3]
    host = [h.reshape(tokens, -1, D) for h in host]
    positions = rng.integers(0, 50, tokens).astype(np.int32)
    if tokens > 4:
        positions[2], positions[3] = -1, 77            # outside the table: not rotated
    angle = rng.uniform(0, 2 * math.pi, (50, rotary // 2))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    weights = [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)] if norm else [None, None]
    pages = 2 * (tokens // page + 2)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 4:
        slots[4] = -1
    if tokens > 5:
        slots[5] = pages * page                        # outside the cache: not written
    return parts, host, positions, cos, sin, weights, pages, slots


@pytest.mark.parametrize("tokens,heads,kv,D,page,rotary,interleaved,norm,dtype,fused", APPENDS)
def test_append_and_read(pn, tokens, heads, kv, D, page, rotary, interleaved, norm, dtype, fused):
    (q, k, v), host, positions, cos, sin, weights, pages, slots = append_case(tokens, heads, kv, D, page, rotary, interleaved,
                                                                              norm, dtype, fused)
    cache = pn.kv_cache(pages, page, kv, D)
    cache.fill_(0xA5)
    want = np.full(tuple(cache.shape), 0xA5, np.uint8)
    table = (cuda(cos), cuda(sin)) if rotary else (None, None)
    got = pn.kv_append(q, k, v, cache, cuda(slots), cuda(positions), *table, q_weight=None if weights[0] is None else cuda(weights[0]),
                       k_weight=None if weights[1] is None else cuda(weights[1]), eps=1e-5, interleaved=interleaved)
    turn = (cos, sin) if rotary else (None, None)
    if heads:
        q_ref = ref.norm_rotate_f32(host[0], weights[0], 1e-5, *turn, positions, interleaved).astype(np.float16)
        assert np.array_equal(got.cpu().numpy(), q_ref)
    else:
        assert got is None
    k_ref = ref.norm_rotate_f32(host[1], weights[1], 1e-5, *turn, positions, interleaved)
    kept = np.where((slots >= 0) & (slots < pages * page), slots, -1)
    kn, kd = ref.quantise(k_ref)
    vn, vd = ref.quantise(host[2].astype(np.float32))
    ref.write_tokens(want, kept, kn, kd, vn, vd)
    assert np.array_equal(cache.cpu().numpy(), want)
    rk, rv = pn.kv_read(cache, cuda(slots))
    for x, n, d in ((rk, kn, kd), (rv, vn, vd)):
        y = np.where((kept >= 0)[:, None, None], ref.dequantise(n, d), 0.0).astype(np.float32)
        assert np.array_equal(x.cpu().numpy(), y)


def test_append_norm_against_64_bits(pn):
    """The normed and rotated queries against the formula in 64 bits: fp32 arithmetic (a dozen
    roundings of 2^-24 and the pairwise sum's eight) is far inside the fp16 rounding of 2^-11."""
    (q, k, v), host, positions, cos, sin, weights, pages, slots = append_case(20, 4, 2, 128, 16, 128, False, True, "f32", False)
    cache = pn.kv_cache(pages, 16, 2, 128)
    got = pn.kv_append(q, k, v, cache, cuda(slots), cuda(positions), cuda(cos), cuda(sin), cuda(weights[0]), cuda(weights[1]), eps=1e-6)
    x = host[0].astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * weights[0]
    for t, p in enumerate(positions):
        if 0 <= p < 50:
            z = (y[t, :, :64] + 1j * y[t, :, 64:]) * (cos[p].astype(np.float64) + 1j * sin[p].astype(np.float64))
            y[t, :, :64], y[t, :, 64:] = z.real, z.imag
    # a rotated value's absolute error goes with its pair's size
    size = np.maximum(np.abs(y), np.sqrt(y[..., :64] ** 2 + y[..., 64:] ** 2).repeat(2, -1).reshape(y.shape[:-1] + (64, 2)).transpose(0, 1, 3, 2).reshape(y.shape))
    assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - y) <= 2.0 ** -11 * np.abs(y) + 2.0 ** -19 * size + 2.0 ** -25)


def test_append_refusals(pn):
    cache = pn.kv_cache(4, 16, 2, 64)
    k = torch.zeros(3, 2, 64, device="cuda")
    slots = torch.arange(3, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    cos = torch.zeros(5, 32, device="cuda")
    ok = pn.kv_append(k.clone(), k, k.clone(), cache, slots, pos, cos, cos)
    assert ok.shape == (3, 2, 64) and ok.dtype == torch.float16
    with pytest.raises(TypeError):
        pn.kv_append(None, k.double(), k, cache, slots)
    with pytest.raises(TypeError):
        pn.kv_append(None, k, k.half(), cache, slots)
    with pytest.raises(ValueError):
        pn.kv_append(None, k[:, :1], k, cache, slots)
    with pytest.raises(ValueError):
        pn.kv_append(None, k.transpose(1, 2).contiguous().transpose(1, 2), k, cache, slots)
    with pytest.raises(ValueError):
        pn.kv_append(None, k, k, cache, slots[:2])
    with pytest.raises(TypeError):
        pn.kv_append(None, k, k, cache, slots, None, cos, cos)
    with pytest.raises(ValueError):
        pn.kv_append(None, k, k, cache, slots, pos, cos, cos[:4])
    with pytest.raises(pn.PnError) as e:              # more pairs than a head has
        pn.kv_append(None, k, k, cache, slots, pos, torch.zeros(5, 33, device="cuda"), torch.zeros(5, 33, device="cuda"))
    assert e.value.status == 1
    with pytest.raises(pn.PnError) as e:
        pn.kv_append(None, k, k, cache, slots, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        pn.kv_cache(4, 16, 2, 96)
    with pytest.raises(ValueError):
        pn.kv_cache(4, 20, 2, 64)
    none = torch.zeros(0, 2, 64, device="cuda")
    assert pn.kv_append(none, none, none, cache, slots[:0]).shape == (0, 2, 64)
    assert pn.kv_read(cache, slots[:0])[0].shape == (0, 2, 64)


# ---------------------------------------------------------------- attention --
def attention_case(lens, counts, heads, kv, D, page, seed=0, k_size=1.0, v_size=1.0, spare_rows=0, fill=0xFF):
    """Cached tokens with known values; every byte that holds no token is 0xFF (NaN scales; `fill`), and
    table entries behind a request's pages lie outside the cache."""
    rng = np.random.default_rng(seed + D + sum(lens))
    held = [-(-x // page) for x in lens]
    pages = sum(held) + 2
    order = rng.permutation(pages)
    table = np.full((len(lens), max(max(held), 1) + 1), 1 << 30, np.int32)
    cache = np.full((pages, kv, page // 16, 17 * D), fill, np.uint8)
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        own = order[at:at + held[b]]
        at += held[b]
        if n == 0:
            ks.append(np.zeros((0, kv, D)))
            vs.append(np.zeros((0, kv, D)))
            continue
        table[b, :held[b]] = own
        k = (k_size * rng.standard_normal((n, kv, D))).astype(np.float32)
        v = (v_size * rng.standard_normal((n, kv, D)) * 2.0 ** rng.integers(-2, 3, (n, 1, 1))).astype(np.float32)
        if n > 3:
            v[3] = 0                                  # a token whose values are all zero
        kn, kd = ref.quantise(k)
        vn, vd = ref.quantise(v)
        slots = [own[t // page] * page + t % page for t in range(n)]
        ref.write_tokens(cache, slots, kn, kd, vn, vd)
        ks.append(ref.dequantise(kn, kd))
        vs.append(ref.dequantise(vn, vd))
    T = sum(counts) + spare_rows
    q = rng.standard_normal((T, heads, D)).astype(np.float16)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return q, cache, table, np.array(lens, np.int32), starts, ks, vs


def check_attention(pn, case, max_queries, scale, window=0, sinks=0, workspace=None, q=None):
    q_host, cache, table, lens, starts, ks, vs = case
    q_dev = cuda(q_host) if q is None else q
    out, lse = pn.attention(q_dev, cuda(cache), cuda(table), cuda(lens), cuda(starts), max_queries, scale, window=window, sinks=sinks,
                            return_lse=True, workspace=workspace)
    if workspace is not None:
        assert workspace.status() == 0
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b in range(len(lens)):
        rows = slice(starts[b], starts[b + 1])
        if starts[b] == starts[b + 1]:
            continue
        want, want_lse, size, reach = ref.attention(q_host[rows].astype(np.float64), ks[b], vs[b], scale, window, sinks)
        L = len(ks[b])
        e = 2.0 ** -19 * reach + 2.0 ** -22 * (1.5 * np.maximum(reach, 10) + 14) + 2.0 ** -21 + L * 2.0 ** -24
        big = np.abs(vs[b]).max() if L else 0.0
        limit = (2.0 ** -11 + 2 * e)[..., None] * size + L * 2.0 ** -35 * big + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
        # beyond fp16 (65520 rounds to infinity) an output is infinite, at its edge it may be
        over = np.abs(want) - limit >= 65520
        edge = np.abs(want) + limit >= 65520
        assert np.array_equal(out[rows][over], np.sign(want[over]) * np.inf), f"request {b}"
        assert np.isfinite(out[rows][~edge]).all(), f"request {b}"
        near = np.abs(np.where(edge, want, out[rows]) - want) <= limit
        assert np.all(near), f"request {b}: {np.abs(out[rows] - want)[~near].max()}"
        none = np.isinf(want_lse)
        assert np.array_equal(none, np.isinf(lse[rows])) and np.all(lse[rows][none] < 0)
        assert np.all(out[rows][none] == 0)
        d = np.abs(lse[rows][~none] - want_lse[~none])
        assert np.all(d <= (2 * e + 2.0 ** -22 * np.abs(want_lse))[~none]), f"request {b}"
    return out, lse


ATTENTIONS = [
    # lens, queries of each, heads, kv heads, D, page, window, sinks
    ([1], [1], 1, 1, 64, 16, 0, 0), ([1], [1], 8, 1, 128, 16, 0, 0), ([1], [1], 6, 1, 256, 16, 0, 0),
    ([15, 16, 17], [1, 1, 1], 4, 2, 128, 16, 0, 0), ([63, 64, 65, 0, 130], [1, 1, 1, 1, 1], 8, 2, 64, 32, 0, 0),
    ([200, 1, 77], [1, 1, 1], 10, 2, 256, 64, 0, 0), ([1000], [1], 16, 4, 128, 128, 0, 0),
    ([2500, 3], [1, 1], 8, 8, 128, 16, 0, 0), ([1500, 700], [1, 1], 24, 2, 128, 64, 0, 0),
    # drafts: several queries of each request, ragged, more queries than tokens, none
    ([40, 3, 64, 9], [4, 3, 0, 4], 4, 2, 128, 16, 0, 0), ([100, 2], [8, 8], 6, 1, 128, 32, 0, 0),
    ([333, 90], [7, 5], 12, 2, 64, 16, 0, 0), ([129, 500], [3, 16], 10, 2, 256, 16, 0, 0),
    # windows and first tokens
    ([500, 20, 64], [1, 1, 1], 4, 1, 128, 16, 100, 4), ([700], [1], 4, 4, 64, 64, 1, 0), ([700], [1], 8, 2, 256, 32, 64, 70),
    ([900, 350], [8, 3], 12, 2, 128, 16, 130, 17), ([300], [5], 2, 1, 128, 16, 1, 1), ([260], [1], 4, 1, 128, 16, 10000, 3),
    # prompts
    ([70], [70], 4, 2, 128, 16, 0, 0), ([200, 150], [130, 150], 6, 2, 64, 32, 0, 0), ([290], [257], 5, 1, 256, 64, 0, 0),
    ([400], [300], 4, 1, 128, 16, 90, 5), ([333, 40, 129], [200, 40, 1], 8, 1, 128, 64, 0, 0),
    ([130], [130], 3, 3, 256, 128, 33, 70), ([270], [270], 2, 2, 64, 16, 64, 0),
]


@pytest.mark.parametrize("lens,counts,heads,kv,D,page,window,sinks", ATTENTIONS)
def test_attention(pn, lens, counts, heads, kv, D, page, window, sinks):
    case = attention_case(lens, counts, heads, kv, D, page)
    ws = pn.AttentionWorkspace()
    first = check_attention(pn, case, max(max(counts), 1), 1 / math.sqrt(D), window, sinks, ws)
    again = check_attention(pn, case, max(max(counts), 1), 1 / math.sqrt(D), window, sinks, ws)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("k_size,v_size,scale", [(30.0, 1.0, 0.3), (1e-3, 1e-4, 0.1), (1.0, 3e4, -0.1), (2.0, 1e-7, 1.0), (1.0, 1.0, 0.0)])
def test_attention_sizes_of_values(pn, D, k_size, v_size, scale):
    """Sharp and flat softmax, scales of V from fp16's subnormals to near its largest, scale <= 0."""
    for counts in ([1, 1], [9, 20]):
        check_attention(pn, attention_case([150, 33], counts, 4, 2, D, 16, 1, k_size, v_size), max(counts), scale)


@pytest.mark.parametrize("counts", [[1] * 3, [40] * 3])
def test_attention_hidden_bytes(pn, counts):
    """Pages outside the cache hide their tokens; a later token's NaN or infinite scale does not reach an earlier query."""
    D, page, kv = 128, 16, 1
    q, cache, table, lens, starts, ks, vs = attention_case([100, 60, 45], counts, 4, kv, D, page)
    # request 0 loses pages 1 and 4: rebuild its reference without those tokens by giving them no weight
    lost = [t for t in range(100) if t // page in (1, 4)]
    table[0, 1], table[0, 4] = -3, cache.shape[0]
    ws = pn.AttentionWorkspace()
    out, lse = pn.attention(cuda(q), cuda(cache), cuda(table), cuda(lens), cuda(starts), max(counts), 0.1, return_lse=True, workspace=ws)
    assert ws.status() == 0
    out = out.cpu().numpy().astype(np.float64)
    n = counts[0]
    for i in range(n):
        p = 100 - n + i
        t = np.array([x for x in range(p + 1) if x not in lost])
        for h in range(4):
            x = 0.1 * ks[0][t, 0] @ q[i, h].astype(np.float64)
            w = np.exp(x - x.max())
            w /= w.sum()
            want = w @ vs[0][t, 0]
            limit = 2.0 ** -10 * (w @ np.abs(vs[0][t, 0])) + 2.0 ** -11 * np.abs(want) + 1e-6
            assert np.all(np.abs(out[i, h] - want) <= limit)
    # the last token of request 1 gets NaN and infinite scales: only its own (last) query sees it
    if n > 1:
        slot = int(table[1, 59 // page]) * page + 59 % page
        rec = cache[slot // page, 0, slot % page // 16]
        r = slot % 16
        for base, bits in ((8 * D, 0x7C00), (16 * D + D // 2, 0x7E00)):
            rec[base + 4 * r: base + 4 * r + 4] = np.array([bits, bits], np.uint16).view(np.uint8)
        got = pn.attention(cuda(q), cuda(cache), cuda(table), cuda(lens), cuda(starts), max(counts), 0.1).cpu().numpy().astype(np.float64)
        rows = slice(starts[1], starts[2] - 1)
        assert np.isfinite(got[rows]).all()
        assert np.array_equal(got[rows], out[rows])
        assert np.isnan(got[starts[2] - 1]).any()


def test_attention_long_and_split(pn):
    """One request over every thread block, lengths around the block boundaries, against its parts:
    the values of a long cache are one page's tokens over and over, so 64 bits need only that page."""
    D, kv, heads, page = 128, 2, 8, 64
    rng = np.random.default_rng(3)
    k = rng.standard_normal((page, kv, D)).astype(np.float32)
    v = (1 + rng.standard_normal((page, kv, D))).astype(np.float32)
    kn, kd = ref.quantise(k)
    vn, vd = ref.quantise(v)
    cache = np.full((2, kv, page // 16, 17 * D), 0xFF, np.uint8)
    ref.write_tokens(cache, list(range(page)), kn, kd, vn, vd)
    kf, vf = ref.dequantise(kn, kd), ref.dequantise(vn, vd)
    q = rng.standard_normal((1, heads, D)).astype(np.float16)
    ws = pn.AttentionWorkspace()
    for length in (4096, 19456, 19457, 70000, 200001):
        table = np.zeros((1, -(-length // page)), np.int32)
        out, lse = pn.attention(cuda(q), cuda(cache), cuda(table), cuda(np.array([length], np.int32)), cuda(np.array([0, 1], np.int32)),
                                1, 0.1, return_lse=True, workspace=ws)
        assert ws.status() == 0
        times = np.full(page, length // page) + (np.arange(page) < length % page)
        for h in range(heads):
            x = 0.1 * kf[:, h // 4] @ q[0, h].astype(np.float64)
            w = times * np.exp(x - x.max())
            want_lse = x.max() + np.log(w.sum())
            w /= w.sum()
            want, size = w @ vf[:, h // 4], w @ np.abs(vf[:, h // 4])
            e = 2.0 ** -19 * 20 + 2.0 ** -22 * 44 + 2.0 ** -21 + length * 2.0 ** -24
            assert np.all(np.abs(out[0, h].cpu().numpy().astype(np.float64) - want)
                          <= (2.0 ** -11 + 2 * e) * size + length * 2.0 ** -35 * 8 + 2.0 ** -11 * np.abs(want))
            assert abs(float(lse[0, h]) - want_lse) <= 2 * e + 2.0 ** -22 * abs(want_lse)


def test_attention_strides_streams_and_rows(pn):
    """Queries as a slice of wider rows, rows of no request left alone, a stream of one's own, no workspace given."""
    case = attention_case([90, 40], [3, 2], 4, 2, 128, 16, spare_rows=2)
    q_host, cache, table, lens, starts, ks, vs = case
    wide = torch.full((7, 4 * 128 + 24), float("nan"), dtype=torch.float16, device="cuda")
    q = wide[:, 8:8 + 512].unflatten(1, (4, 128))
    q.copy_(torch.from_numpy(q_host))
    plain, _ = check_attention(pn, case, 3, 0.1)
    args = [cuda(x) for x in (cache, table, lens, starts)]
    out = torch.full((7, 4, 128), 7.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pn.attention(q, *args, 3, 0.1, out=out, stream=side)
    side.synchronize()
    assert np.array_equal(out[:5].cpu().numpy().astype(np.float64), plain[:5])
    assert torch.all(out[5:] == 7.0)


def test_attention_refusals(pn):
    q, cache, table, lens, starts = (cuda(x) for x in attention_case([20], [1], 4, 2, 64, 16)[:5])
    ws = pn.AttentionWorkspace()
    good = (q, cache, table, lens, starts, 1, 0.1)
    pn.attention(*good, workspace=ws)

    def status(*args, **kw):
        with pytest.raises(pn.PnError) as e:
            pn.attention(*args, workspace=ws, **kw)
        return e.value.status

    assert status(q[:, :3], *good[1:]) == 1                           # heads no multiple of kv heads
    assert status(*good[:5], 0, 0.1) == 1
    assert status(*good[:6], float("nan")) == 1
    assert status(*good, window=-1) == 1
    assert status(*good, sinks=-1) == 1
    assert status(*good, out=q) == 1                                  # output over input
    shifted = torch.zeros(4 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(1, 4, 64)
    assert status(shifted, *good[1:]) == 2
    with pytest.raises(TypeError):
        pn.attention(q.float(), *good[1:])
    with pytest.raises(TypeError):
        pn.attention(q, cache, table.long(), *good[3:])
    with pytest.raises(ValueError):
        pn.attention(q, cache, table, lens, starts[:1], 1, 0.1)
    with pytest.raises(ValueError):
        pn.attention(q[:, :, :32], *good[1:])
    assert pn.attention(q[:0], cache, table, lens, torch.zeros(2, dtype=torch.int32, device="cuda"), 1, 0.1, workspace=ws).shape == (0, 4, 64)


@pytest.mark.parametrize("counts", [[1], [40]])
def test_attention_time_out(pn, counts):
    """A copy that never comes ends in PN_ETIMEOUT, and the workspace serves the next call."""
    case = attention_case([300], counts, 4, 2, 128, 16)
    ws = pn.AttentionWorkspace()
    args = [cuda(x) for x in case[:5]]
    pn.set_wait_timeout_ns(2_000_000)
    pn.set_test_stall(True)
    try:
        pn.attention(*args, counts[0], 0.1, workspace=ws)
        assert ws.status() == 5
    finally:
        pn.set_test_stall(False)
        pn.set_wait_timeout_ns(1_000_000_000)
    check_attention(pn, case, counts[0], 0.1, workspace=ws)


# ------------------------------------------------------------------- verify --
def probabilities(rng, shape, sharp):
    x = sharp * rng.standard_normal(shape)
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


VERIFIES = [(1, 0, 5, 1.0, True), (1, 1, 1, 1.0, False), (3, 3, 33, 1.0, False), (9, 7, 1000, 3.0, False), (9, 7, 1000, 3.0, True),
            (40, 5, 257, 0.1, False), (5, 31, 64, 2.0, True), (4, 15, 32001, 2.0, False), (2, 3, 151936, 4.0, False), (300, 2, 100, 1.0, False)]


@pytest.mark.parametrize("batch,drafts,vocab,sharp,certain", VERIFIES)
@pytest.mark.parametrize("counted", [False, True])
def test_verify(pn, batch, drafts, vocab, sharp, certain, counted):
    rng = np.random.default_rng(batch + vocab)
    target = probabilities(rng, (batch, drafts + 1, vocab), sharp)
    draft = None
    if not certain:
        draft = target[:, :drafts] * rng.uniform(0.3, 1.7, (batch, drafts, vocab)).astype(np.float32)
        draft = (draft / draft.sum(-1, keepdims=True)).astype(np.float32) if drafts else draft
    tokens = target[:, :drafts].argmax(-1).astype(np.int32)
    if drafts and batch > 2:
        tokens[1, 0], tokens[2, drafts - 1] = -1, vocab               # outside the vocabulary
    uniforms = rng.random((batch, drafts + 1)).astype(np.float32)
    uniforms[0, -1] = 0.0
    uniforms[-1, -1] = np.nextafter(np.float32(1), np.float32(0))
    counts = rng.integers(0, drafts + 1, batch).astype(np.int32) if counted else None
    got = pn.verify(cuda(tokens), cuda(target), None if draft is None else cuda(draft), cuda(uniforms),
                    counts=None if counts is None else cuda(counts))
    want = ref.verify(tokens, target, draft, uniforms, counts)
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert np.array_equal(got[1].cpu().numpy(), want[1])


def test_verify_rows_with_nothing(pn):
    """Equal rows (nothing left of p - q), rows of zeros and NaN, one certain token, weights above one."""
    V, K = 700, 2
    target = np.zeros((6, K + 1, V), np.float32)
    draft = np.zeros((6, K, V), np.float32)
    target[0, :, 5:9] = 0.25
    draft[0] = target[0, :K]                                          # u = 0.9999 * 0.25 < 0.25: all accepted
    target[1, 0, 3], draft[1, 0, 3] = 0.5, 1.0                        # turned down, p - q leaves nothing: p itself
    target[2] = 0                                                     # a row of zeros
    target[3] = np.nan
    target[4, :, 699] = 1.0
    target[5, :, ::2] = 3.0
    tokens = np.array([[5, 6], [3, 3], [1, 1], [1, 1], [699, 0], [1, 1]], np.int32)
    uniforms = np.full((6, K + 1), 0.75, np.float32)
    got = pn.verify(cuda(tokens), cuda(target), cuda(draft), cuda(uniforms))
    want = ref.verify(tokens, target, draft, uniforms, None)
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert want[1][1].tolist() == [3, -1, -1] and want[1][2].tolist() == [-1, -1, -1]


def test_verify_refusals(pn):
    t = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    p = torch.zeros(2, 4, 10, device="cuda")
    u = torch.zeros(2, 4, device="cuda")
    pn.verify(t, p, None, u)
    with pytest.raises(ValueError):
        pn.verify(t, p[:, :3].contiguous(), None, u)
    with pytest.raises(ValueError):
        pn.verify(t, p, p, u)
    with pytest.raises(TypeError):
        pn.verify(t, p.half(), None, u)
    with pytest.raises(pn.PnError) as e:
        pn.verify(torch.zeros(1, 32, dtype=torch.int32, device="cuda"), torch.zeros(1, 33, 4, device="cuda"), None,
                  torch.zeros(1, 33, device="cuda"))
    assert e.value.status == 1
    a, o = pn.verify(t[:0], p[:0], None, u[:0])
    assert a.shape == (0,) and o.shape == (0, 4)


# ------------------------------------------------- large batches, far addresses --
@pytest.mark.parametrize("batch,D,queries", [(9001, 128, 1), (16384, 128, 1), (16384, 64, 12), (16384, 256, 1), (16384, 128, 60)])
def test_attention_many_requests(pn, batch, D, queries):
    """Batches whose prefix sums take shared memory from the stages: one request in eight has 1 to 3 tokens, the last `queries`."""
    rng = np.random.default_rng(batch + D)
    lens = rng.integers(1, 4, batch) * (rng.random(batch) < 0.125)
    lens[-1] = 70
    counts = [int(x > 0) for x in lens]
    counts[-1] = queries
    case = attention_case([int(x) for x in lens], counts, 2, 1, D, 16)
    ws = pn.AttentionWorkspace()
    check_attention(pn, case, queries, 1 / math.sqrt(D), workspace=ws)


@pytest.mark.parametrize("D,queries", [(128, 1), (128, 8), (128, 70), (256, 3)])
def test_far_pages(pn, D, queries):
    """A cache of more than 2^32 bytes: what is written to its last pages reads back, and attends, as in a small one."""
    kv, heads, page, tokens = 8, 16, 1024, 1500
    page_bytes = kv * page // 16 * 17 * D
    pages = (1 << 32) // page_bytes + 40
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v = (torch.randn(tokens, h, D, device="cuda", generator=g) for h in (heads, kv, kv))
    place = torch.arange(tokens, device="cuda")
    near, far = pn.kv_cache(2, page, kv, D), pn.kv_cache(pages, page, kv, D)
    q_near = pn.kv_append(q, k, v, near, place)
    q_far = pn.kv_append(q, k, v, far, place + (pages - 2) * page)
    assert torch.equal(q_near, q_far)
    for a, b in zip(pn.kv_read(near, place), pn.kv_read(far, place + (pages - 2) * page)):
        assert torch.equal(a, b)
    assert not far[:pages - 2].any()
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
    tables = [torch.tensor([[p, p + 1]], dtype=torch.int32, device="cuda") for p in (0, pages - 2)]
    got = [pn.attention(q_near[-queries:], c, t, lens, starts, queries, 0.1, return_lse=True) for c, t in zip((near, far), tables)]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_attention_too_many_units(pn):
    """Shapes whose bound on the work passes 32 bits are refused before anything is launched."""
    q, cache, table, lens, starts = (cuda(x) for x in attention_case([20], [1], 8, 8, 256, 16)[:5])
    many = torch.zeros(16384, dtype=torch.int32, device="cuda")
    table = torch.zeros(16384, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(pn.PnError) as e:             # 16384 requests, 8 heads, 2^14 groups of 8 rows: a unit and one more for each
        pn.attention(q, cache, table, many, torch.zeros(16385, dtype=torch.int32, device="cuda"), 1 << 17, 0.1)
    assert e.value.status == 3


@pytest.mark.parametrize("vocab", [(1 << 20) - 3, 1 << 20])
def test_verify_largest_vocabulary(pn, vocab):
    """Weights of 1 and above in every place: the sums at their bound."""
    target = np.full((2, 2, vocab), 1.0, np.float32)
    target[1] = 2.0
    target[1, :, ::3] = 0.7
    tokens = np.array([[3], [vocab - 1]], np.int32)
    uniforms = np.array([[0.5, 0.9999], [0.5, 0.31]], np.float32)
    got = pn.verify(cuda(tokens), cuda(target), None, cuda(uniforms))
    want = ref.verify(tokens, target, None, uniforms, None)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


def test_plan_counts_past_32_bits(pn):
    """Tokens whose sum passes 2^31 and 2^32 are refused, those before them served."""
    big = (1 << 31) - 1
    lens = torch.tensor([3, big, 0, big, 1], dtype=torch.int32, device="cuda")
    add = torch.tensor([5, big, big, big, 7], dtype=torch.int32, device="cuda")
    held = torch.tensor([1, 0, 0, 0, 1], dtype=torch.int32, device="cuda")
    table = torch.full((5, 4), 9, dtype=torch.int32, device="cuda")
    free, ring = torch.arange(10, dtype=torch.int32, device="cuda"), torch.tensor([(1 << 40) + 2, (1 << 40) + 8], device="cuda")
    p = pn.kv_plan(lens, add, held, table, free, ring, 16, 40)
    assert p.starts.tolist() == [0, 5] + [(1 << 31) - 16] * 4
    assert p.lens.tolist() == [8, big, 0, big, 1] and p.held.tolist() == [1, 0, 0, 0, 1]
    assert p.refused.tolist() == [4] and p.ring.tolist() == ring.tolist()
    assert p.slots.tolist() == [9 * 16 + 3 + i for i in range(5)] + [-1] * 35
    assert p.requests.tolist() == [0] * 5 + [1] * 35 and p.positions.tolist() == [3, 4, 5, 6, 7] + [-1] * 35


# ------------------------------------------- many query rows (products on tcgen05) --
MANY_ROWS = [
    # lens, queries of each, heads, kv heads, D, page, window, sinks
    ([401], [384], 8, 8, 64, 16, 0, 0), ([390], [384], 8, 8, 128, 64, 0, 0), ([385], [384], 8, 8, 256, 32, 0, 0),
    ([130, 77, 500], [120, 77, 130], 48, 8, 128, 16, 0, 0), ([140, 333], [140, 100], 40, 8, 256, 128, 0, 0),
    ([129, 300], [128, 200], 56, 8, 64, 64, 0, 0),
    ([700], [400], 16, 8, 128, 32, 100, 5), ([640], [400], 16, 8, 256, 16, 33, 70), ([600, 90], [300, 90], 16, 8, 64, 16, 1, 1),
    ([40] * 30 + [0, 3, 200], [40] * 30 + [0, 3, 40], 12, 3, 128, 16, 0, 0), ([33] * 40, [33] * 40, 8, 2, 256, 16, 20, 3),
    ([2000], [390], 8, 8, 256, 64, 0, 0), ([3000], [390], 8, 8, 128, 16, 0, 0),
]


@pytest.mark.parametrize("lens,counts,heads,kv,D,page,window,sinks", MANY_ROWS)
def test_attention_many_rows(pn, lens, counts, heads, kv, D, page, window, sinks):
    case = attention_case(lens, counts, heads, kv, D, page)
    ws = pn.AttentionWorkspace()
    first = check_attention(pn, case, max(counts), 1 / math.sqrt(D), window, sinks, ws)
    again = check_attention(pn, case, max(counts), 1 / math.sqrt(D), window, sinks, ws)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("k_size,v_size,scale", [(30.0, 1.0, 0.3), (1e-3, 1e-4, 0.1), (1.0, 3e4, -0.1), (2.0, 1e-7, 1.0), (1.0, 1.0, 0.0)])
def test_attention_many_rows_sizes_of_values(pn, D, k_size, v_size, scale):
    case = attention_case([150, 133], [128, 128], 24, 8, D, 16, 1, k_size, v_size)
    check_attention(pn, case, 128, scale)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_many_rows_hidden_bytes(pn, D):
    """Lost pages hide their tokens; a last token's NaN and infinite scales reach its own query alone."""
    B, L, n, page = 34, 100, 40, 16
    q, cache, table, lens, starts, ks, vs = attention_case([L] * B, [n] * B, 4, 1, D, page)
    for b in range(0, B, 3):
        table[b, 1], table[b, 4] = -3, cache.shape[0]
    run = lambda: pn.attention(cuda(q), cuda(cache), cuda(table), cuda(lens), cuda(starts), n, 0.1).cpu().numpy().astype(np.float64)
    out = run()
    for b in (0, 1, 33):
        lost = [t for t in range(L) if t // page in (1, 4)] if b % 3 == 0 else []
        for i in (0, 5, n - 1):
            t = np.array([x for x in range(L - n + i + 1) if x not in lost])
            for h in range(4):
                x = 0.1 * ks[b][t, 0] @ q[starts[b] + i, h].astype(np.float64)
                w = np.exp(x - x.max())
                w /= w.sum()
                want = w @ vs[b][t, 0]
                limit = 2.0 ** -10 * (w @ np.abs(vs[b][t, 0])) + 2.0 ** -11 * np.abs(want) + 1e-6
                assert np.all(np.abs(out[starts[b] + i, h] - want) <= limit)
    NG = D // 64
    for b in range(1, B, 3):
        slot = int(table[b, (L - 1) // page]) * page + (L - 1) % page
        rec, r = cache[slot // page, 0, slot % page // 16], slot % 16
        for base, bits in ((8 * D, 0x7C00), (16 * D + D // 2, 0x7E00)):
            rec[base + 2 * NG * r: base + 2 * NG * (r + 1)] = np.array([bits] * NG, np.uint16).view(np.uint8)
    got = run()
    last = np.zeros(len(q), bool)
    last[starts[2::3] - 1] = True                     # the last queries of requests 1, 4, ...
    assert np.array_equal(got[~last], out[~last])
    assert all(np.isnan(got[i]).any() for i in np.flatnonzero(last))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_many_rows_time_out(pn, D):
    """A copy that never comes ends in the status word, and the workspace serves the next call."""
    case = attention_case([400], [384], 8, 8, D, 16)
    args = [cuda(x) for x in case[:5]]
    ws = pn.AttentionWorkspace()
    pn.set_wait_timeout_ns(20_000_000)
    pn.set_test_stall(True)
    try:
        pn.attention(*args, 384, 0.1, workspace=ws)
        assert ws.status() == 5
    finally:
        pn.set_test_stall(False)
        pn.set_wait_timeout_ns(1_000_000_000)
    check_attention(pn, case, 384, 0.1, workspace=ws)


def test_attention_many_requests_and_rows(pn):
    """16384 requests, most empty, the last with many rows: prefix sums of a large batch."""
    lens = [0] * 16384
    counts = [0] * 16384
    for b, n in ((0, 3), (5000, 70), (16383, 200)):
        lens[b], counts[b] = n + 10, n
    check_attention(pn, attention_case(lens, counts, 4, 2, 128, 16), 200, 0.1, workspace=pn.AttentionWorkspace())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,counts,heads,kv", [([70, 3, 45], [1, 1, 1], 4, 2), ([70, 41, 29], [12, 3, 9], 4, 2), ([171, 141], [160, 140], 24, 8)])
@pytest.mark.parametrize("v_size", [1.0, 1e-4])
def test_attention_stale_bytes(pn, D, lens, counts, heads, kv, v_size):
    """What bytes behind the last token hold (large finite scales, infinite ones, zeros) changes no bit."""
    runs = []
    for fill in (0x00, 0x7B, 0x7C, 0xFF):
        case = attention_case(lens, counts, heads, kv, D, 64, 3, 1.0, v_size, fill=fill)
        runs.append(check_attention(pn, case, max(counts), 0.1))
    for r in runs[1:]:
        assert np.array_equal(r[0], runs[0][0]) and np.array_equal(r[1], runs[0][1])


# ------------------------------------------------ windows and first tokens near 2^31 --
MOST = (1 << 31) - 1


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,counts,heads,kv", [([500, 40, 3], [1, 3, 1], 4, 2), ([500, 40], [9, 3], 4, 2), ([390, 140], [384, 130], 8, 8)])
@pytest.mark.parametrize("window,sinks", [(100, MOST), (10000, MOST), (1, MOST - 40), (130, MOST - 100), (MOST, 0), (MOST - 7, MOST - 12)])
def test_attention_all_first_tokens(pn, D, lens, counts, heads, kv, window, sinks):
    """As many first tokens as can be asked for, or such a window, hide nothing."""
    case = attention_case(lens, counts, heads, kv, D, 16)
    got = check_attention(pn, case, max(counts), 0.1, window, sinks, pn.AttentionWorkspace())
    plain = check_attention(pn, case, max(counts), 0.1)
    if window >= 10000:                               # more than the table has room for: the same call, so the same bits
        assert np.array_equal(got[0], plain[0]) and np.array_equal(got[1], plain[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,counts,heads,kv", [([2, 9, 1], [5, 16, 1], 4, 2), ([100, 2, 250], [384, 30, 384], 8, 8)])
@pytest.mark.parametrize("window,sinks", [(MOST, 0), (MOST - 3, MOST), (5, MOST), (MOST, MOST), (90, 3)])
def test_attention_more_queries_than_tokens_and_windows(pn, D, lens, counts, heads, kv, window, sinks):
    """Queries before the cache see nothing, those behind them what their window and the first tokens hold."""
    case = attention_case(lens, counts, heads, kv, D, 16)
    check_attention(pn, case, max(counts), 0.1, window, sinks, pn.AttentionWorkspace())


# ----------------------------------- one long prompt among many requests, long tables --
MIXED = [
    # lens, queries of each, max_queries, heads, kv heads, D, page, columns of the table
    ([90] + [7, 33, 64, 1] * 15 + [200, 16, 3], [40] + [1] * 63, 8192, 64, 8, 128, 16, 8192),
    ([300] + [20, 45, 1] * 85, [260] + [1] * 255, 2048, 64, 8, 128, 64, 2048),
    ([70] + [5, 17] * 40, [33] + [1] * 80, 8192, 64, 8, 256, 16, 8192), ([70] + [5, 17] * 40, [33] + [1] * 80, 8192, 64, 8, 64, 16, 8192),
    ([0] * 16000 + [30, 9, 77] + [0] * 381, [0] * 16000 + [1, 1, 48] + [0] * 381, 48, 8, 8, 64, 1024, 512),
]


@pytest.mark.parametrize("lens,counts,most,heads,kv,D,page,columns", MIXED)
def test_attention_long_tables(pn, lens, counts, most, heads, kv, D, page, columns):
    """The bound on the work goes by the queries that there are, not by max_queries for every request."""
    q, cache, table, lens, starts, ks, vs = attention_case(lens, counts, heads, kv, D, page)
    wide = np.full((len(lens), columns), 1 << 30, np.int32)
    wide[:, :table.shape[1]] = table
    check_attention(pn, (q, cache, wide, lens, starts, ks, vs), most, 1 / math.sqrt(D), workspace=pn.AttentionWorkspace())


@pytest.mark.parametrize("D,queries,kv", [(256, 32, 8), (128, 8192, 8)])
def test_attention_starts_out_of_order(pn, D, queries, kv):
    """Starts that go up and down make more work than any in order; past 32 bits the call ends at once, and says so."""
    B, page, columns = 16384, 1024, 512
    # 8192 requests x 8 heads x 4 groups of 8 rows x (16383 + 1) units = 2^32; 8192 x 8 x 64 tiles of 128 rows x 8192 of 64 tokens = 2^35
    length = page * columns - (32 if D == 256 else 0)
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = queries
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    cache, ws = pn.kv_cache(1, page, kv, D), pn.AttentionWorkspace()
    q = torch.ones(queries, kv, D, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 7.0)
    pn.attention(q, cache, table, lens, starts, queries, 0.1, out=out, workspace=ws)
    assert ws.status() == 1
    assert torch.all(out == 7.0)
    case = attention_case([40, 9], [3, 1], 4, 2, 64, 16)
    check_attention(pn, case, 3, 0.1, workspace=ws)


# ------------------------------------------------------------- workspace, memory --
@pytest.mark.parametrize("counts", [[1], [200]])
def test_attention_workspace_on_another_stream(pn, counts):
    """A workspace made while the current stream is busy serves a call on another one at once: its zeros are there."""
    case = attention_case([3000], counts, 8, 8, 128, 16)
    q, cache, table, lens, starts = (cuda(x) for x in case[:5])
    plain, plain_lse = pn.attention(q, cache, table, lens, starts, counts[0], 0.1, return_lse=True)
    used = torch.full((pn.AttentionWorkspace().nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del used                                          # the next allocation of this size finds these bytes
    torch.cuda._sleep(100_000_000)
    ws = pn.AttentionWorkspace()
    assert torch.cuda.current_stream().query()
    out, lse = pn.attention(q, cache, table, lens, starts, counts[0], 0.1, return_lse=True, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse) and ws.status() == 0


def test_attention_in_a_graph_without_a_workspace(pn):
    """Captured with a workspace of its own: nothing waits, and every replay gives the call's output."""
    case = attention_case([700, 90], [3, 2], 4, 2, 128, 16)
    q, cache, table, lens, starts = (cuda(x) for x in case[:5])
    plain = pn.attention(q, cache, table, lens, starts, 3, 0.1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = pn.attention(q, cache, table, lens, starts, 3, 0.1)
        ws = pn.AttentionWorkspace()
        again = pn.attention(q, cache, table, lens, starts, 3, 0.1, workspace=ws)
    for _ in range(2):
        out.zero_()
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain) and torch.equal(again, plain)


def test_out_of_memory_is_pytorchs(pn):
    """Outputs past the device's memory (2 x 550 GB) end in the error that PyTorch's own calls raise, and the call works afterwards."""
    cache, slots = pn.kv_cache(1, 16, 65536, 256), torch.zeros(8192, dtype=torch.int64, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        pn.kv_read(cache, slots)
    assert pn.kv_read(cache, slots[:1])[0].shape == (1, 65536, 256)


# ------------------------------------------------- V scales that differ within a tile --
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("counts,heads,kv,rounding", [([3, 2], 4, 2, 2.0 ** -35), ([128, 128], 24, 8, 2.0 ** -32)])
@pytest.mark.parametrize("spread", [1.0, 1e3, 1e6])
@pytest.mark.parametrize("away", [1.0, 4.0])
def test_attention_scales_within_a_tile(pn, D, counts, heads, kv, rounding, spread, away):
    """Every 37th token has values `spread` times the others' and keys that point away from all queries.

    The tolerance is the one at the head of this file but for p_t d_t below fp16's normal numbers, which
    are rounded to 2^-25 each, times |n - 8| <= 8, over the sum of the weights.  For few rows the reference
    keeps the largest p_t d_t at 2^13 or more, so the sum is at least 2^13 over the largest V scale: 2^-35
    of it to a token.  For many rows the reference lies 7 below the largest score plus the largest scale of
    its tile or, in later tiles, lower; so the largest weight, and with it the sum, is at least 2^7 over the
    largest scale: 2^-29 of that, which is 2^-32 of the largest value (eight steps of its scale)."""
    rng = np.random.default_rng(D + int(away))
    page, lens = 32, [400, 333]
    held = [-(-n // page) for n in lens]
    order = rng.permutation(sum(held))
    table = np.full((2, max(held)), 1 << 30, np.int32)
    cache = np.full((sum(held), kv, page // 16, 17 * D), 0xFF, np.uint8)
    side = rng.choice([-1.0, 1.0], (kv, D))
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        own = order[at:at + held[b]]
        at += held[b]
        table[b, :held[b]] = own
        k = (0.5 * rng.standard_normal((n, kv, D))).astype(np.float32)
        v = (1e-2 * rng.standard_normal((n, kv, D))).astype(np.float32)
        k[5::37] = -away * side
        v[5::37] *= spread
        kn, kd = ref.quantise(k)
        vn, vd = ref.quantise(v)
        ref.write_tokens(cache, [own[t // page] * page + t % page for t in range(n)], kn, kd, vn, vd)
        ks.append(ref.dequantise(kn, kd))
        vs.append(ref.dequantise(vn, vd))
    q = (side[:, None] + 0.3 * rng.standard_normal((sum(counts), kv, heads // kv, D))).reshape(-1, heads, D).astype(np.float16)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    scale = 1 / math.sqrt(D)
    ws = pn.AttentionWorkspace()
    out, lse = pn.attention(cuda(q), cuda(cache), cuda(table), cuda(np.array(lens, np.int32)), cuda(starts), max(counts), scale,
                            return_lse=True, workspace=ws)
    assert ws.status() == 0
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b, L in enumerate(lens):
        rows = slice(starts[b], starts[b + 1])
        want, want_lse, size, reach = ref.attention(q[rows].astype(np.float64), ks[b], vs[b], scale, 0, 0)
        e = 2.0 ** -19 * reach + 2.0 ** -22 * (1.5 * np.maximum(reach, 10) + 14) + 2.0 ** -21 + L * 2.0 ** -24
        limit = (2.0 ** -11 + 2 * e)[..., None] * size + L * rounding * np.abs(vs[b]).max() + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
        far = np.abs(out[rows] - want) > limit
        assert not far.any(), f"request {b}: {(np.abs(out[rows] - want) / limit).max()} of the limit"
        assert np.all(np.abs(lse[rows] - want_lse) <= 2 * e + 2.0 ** -22 * np.abs(want_lse)), f"request {b}"
