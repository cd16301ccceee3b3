"""pn_logprobs, pn_norm, pn_kv_weigh and pn_kv_evict against plain restatements in 64 bits.

Tolerances (u = 2^-24, half a step of fp32).

logprobs: e = exp2(d c) errs by 2^-22 of itself for ex2 and by 2 u |d c| for its
argument, which weighted by e / S gives at most 2 u (ln V + 1); a sum takes a chain
of at most V / 8192 + 48 additions (16 and 1 to 32 values, V / 8192 such, 5, 8 and 8
joins with two products each).  With s = (V / 8192 + 64) u + 2^-22 + 2 u (ln V + 1):
  |logprob - exact| <= s + 2^-22 ln V + 2^-22 |x - max x| + 2 u |exact|
  |entropy - exact| <= 2 (ln V + 1) (s + 2^-22)

norm: a sum of squares or of values takes at most 32 + 10 additions, so it errs by 42 u
of the sum of the absolute values; the norm by half of that and 4 u more (quotient,
root, products), the mean by 43 u of mean |v|.  r' takes three roundings more.  An
error in r' moves x's norm by no more than its share of the row's size.

weigh: a probability errs by e = 2^-19 reach + 2^-22 (|x| + |lse| + 2) + 2^-21, reach =
scale sum |q| |k| (as for attention); their sum by a chain of rows / 4 + 12 additions.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HUGE = 1.7e38


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


# ----------------------------------------------------------------- logprobs --
def ref_logprobs(logits, tokens, top, scale):
    """logits [R][V] in 64 bits.  (log probabilities of tokens, entropy, top tokens, their log probabilities, largest x)"""
    R, V = logits.shape
    there = logits > -HUGE                                   # (NaN: no)
    x = np.where(there, np.minimum(np.where(there, logits, 0), HUGE), -np.inf) * scale
    most = x.max(1)
    d = x - np.where(np.isinf(most), 0, most)[:, None]
    e = np.exp(d)
    S = e.sum(1)
    some = S > 0
    log_s = np.log(np.where(some, S, 1))
    log_p = np.where(there, d - log_s[:, None], -np.inf)
    entropy = np.where(some, log_s - np.where(e > 0, e * np.where(e > 0, d, 0), 0).sum(1) / np.where(some, S, 1), 0)
    given = np.full(tokens.shape, -np.inf)
    for r in range(R):
        for i, t in enumerate(tokens[r]):
            if 0 <= t < V:
                given[r, i] = log_p[r, t]
    best, best_p = np.full((R, top), -1, np.int64), np.full((R, top), -np.inf)
    for r in range(R):
        order = sorted(np.flatnonzero(there[r]), key=lambda t: (-logits[r, t], t)) if V <= 4096 else \
            [t for t in np.lexsort((np.arange(V), -np.where(there[r], logits[r], -np.inf)))[:top] if there[r, t]]
        for i, t in enumerate(order[:top]):
            best[r, i], best_p[r, i] = t, log_p[r, t]
    return given, entropy, best, best_p, most


def check_logprobs(pn, logits, tokens, top, scale, device=None):
    """logits: numpy [R][V] of fp32 or fp16; device: the tensor to pass (else a copy of them)."""
    R, V = logits.shape
    got = pn.logprobs(cuda(logits) if device is None else device, cuda(tokens.astype(np.int32)), top=top, scale=scale)
    scale = float(np.float32(scale))
    given, entropy, best, best_p, most = ref_logprobs(logits.astype(np.float64), tokens, top, scale)
    s = (V / 8192 + 64) * U + 2.0 ** -22 + 2 * U * (math.log(V) + 1)

    def near(mine, exact):
        mine = mine.cpu().numpy().astype(np.float64)
        none = np.isinf(exact)
        assert np.array_equal(mine[none], exact[none])
        assert np.isfinite(mine[~none]).all()
        far = np.abs(exact) + math.log(V) + 1                # at least |x - max x|
        limit = s + 2.0 ** -22 * math.log(V) + 2.0 ** -22 * far + 2 * U * np.abs(exact)
        assert np.all(np.abs(mine[~none] - exact[~none]) <= limit[~none]), np.abs(mine[~none] - exact[~none]).max()

    near(got.logprobs.reshape(R, -1), given)
    d = np.abs(got.entropy.cpu().numpy() - entropy)
    assert np.all(d <= 2 * (math.log(V) + 1) * (s + 2.0 ** -22)), d.max()
    if top:
        assert np.array_equal(got.top_tokens.cpu().numpy(), best)
        near(got.top_logprobs, best_p)
    else:
        assert got.top_tokens is None and got.top_logprobs is None
    return got


@pytest.mark.parametrize("rows,vocab,dtype,count,top,scale", [
    (1, 1, "f32", 1, 1, 1.0), (3, 2, "f16", 2, 5, 0.5), (2, 31, "f32", 1, 32, 1.0), (5, 100, "f16", 3, 20, 1.25), (1, 1000, "f32", 1, 1, 2.0),
    (7, 4096, "f16", 1, 32, 1.0), (1, 32000, "f32", 1, 5, 1.0), (3, 50257, "f32", 2, 20, 0.7), (9, 33333, "f16", 1, 7, 1.5), (2, 151936, "f32", 1, 20, 1.0),
    (700, 515, "f32", 1, 3, 1.0), (1, 1 << 20, "f16", 1, 32, 1.0), (2, 20000, "f32", 0, 4, 1.0), (2, 20001, "f16", 1, 0, 1.0), (1300, 4099, "f16", 1, 2, 1.0),
])
def test_logprobs(pn, rows, vocab, dtype, count, top, scale):
    rng = np.random.default_rng(rows * 1000 + vocab)
    logits = (3 * rng.standard_normal((rows, vocab))).astype(np.float32 if dtype == "f32" else np.float16)   # fp16: many ties
    tokens = rng.integers(0, vocab, (rows, count))
    got = check_logprobs(pn, logits, tokens, top, scale)
    again = pn.logprobs(cuda(logits), cuda(tokens.astype(np.int32)), top=top, scale=scale)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("vocab", [5, 300, 8209, 40000])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
def test_logprobs_masks_and_ties(pn, vocab, dtype):
    """Rows without any token, of one token, all equal, in order, of the types' lowest values, infinities and NaN."""
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((13, vocab)).astype(dtype)
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, vocab // 2] = 3
    x[3] = 1.5
    x[4] = np.sort(x[4])
    x[5] = np.sort(x[5])[::-1]
    x[6] = np.finfo(dtype).min
    x[7, ::2] = np.finfo(dtype).min
    x[8, rng.random(vocab) < 0.7] = -np.inf
    x[8, rng.random(vocab) < 0.1] = np.nan
    x[9, :] = 0
    x[9, 1::3] = -0.0                                        # equal to 0
    x[10] = -np.inf
    x[10, -1], x[10, 0] = -2, -2
    x[11, vocab // 3] = np.inf
    x[11, vocab // 3 + 1] = np.inf
    x[12] = 1000 * x[12]
    tokens = np.stack([rng.integers(0, vocab, 13), np.full(13, vocab // 2), np.full(13, -1), np.full(13, vocab), np.full(13, np.iinfo(np.int32).max)], 1)
    check_logprobs(pn, x, tokens, 32, 1.0)
    check_logprobs(pn, x, tokens, 1, 0.3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("offset,width", [(0, 777), (1, 777), (3, 780), (7, 5001)])
def test_logprobs_strides(pn, dtype, offset, width):
    """Rows that begin anywhere in a 16-byte line, with NaN around them."""
    vocab = width - offset - 5
    g = torch.Generator().manual_seed(offset)
    whole = torch.full((6, width), math.nan, dtype=dtype)
    x = torch.randn(6, vocab, generator=g).to(dtype)
    whole[:, offset:offset + vocab] = x
    view = whole.cuda()[:, offset:offset + vocab]
    tokens = np.arange(6)[:, None] * 7 % vocab
    check_logprobs(pn, x.numpy(), tokens, 9, 1.0, device=view)
    one = pn.logprobs(view[2:3], torch.tensor([5], dtype=torch.int32, device="cuda"), top=4)
    assert one.logprobs.shape == (1,) and torch.equal(one.top_tokens, pn.logprobs(view, top=4).top_tokens[2:3])


@pytest.mark.parametrize("order", ["up", "one thread"])
def test_logprobs_top_in_one_place(pn, order):
    """Large values in the order that makes the most work, and all of them where one thread finds them."""
    V = 65536
    x = np.random.default_rng(1).standard_normal((2, V)).astype(np.float32)
    if order == "up":
        x[0] = np.linspace(-5, 5, V, dtype=np.float32)
    else:
        for part in range(8):
            x[0, part * (V // 8) + 40: (part + 1) * (V // 8): 1024] += 100     # every 256th vector of 4
    check_logprobs(pn, x, np.array([[3], [4]]), 32, 1.0)


@pytest.mark.parametrize("rows,vocab,top", [(310, 150001, 32), (310, 150001, 1), (305, 140000, 5), (700, 9001, 20), (3, 4090, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("steps", [0, 4, 300])
def test_logprobs_top_of_whole_rows(pn, rows, vocab, top, dtype, steps):
    """Rows of a block each, long ones among them: the order of a stable sort, with few different values (steps to one) too."""
    torch.manual_seed(rows + top)
    logits = torch.randn(rows, vocab, device="cuda") * 3
    if steps:
        logits = torch.round(logits * steps) / steps
    logits = logits.to(dtype)
    logits[1, :vocab - 3] = -math.inf                        # three tokens left
    logits[2] = 1.5
    got = pn.logprobs(logits, top=top)
    for r in [0, 1, 2, *range(3, rows, 61)]:
        x = logits[r].double()
        order = torch.sort(x, descending=True, stable=True).indices[:top]
        left = min(top, int(torch.isfinite(x).sum()))
        assert torch.equal(got.top_tokens[r, :left].long(), order[:left]) and (got.top_tokens[r, left:] == -1).all(), r
        want = x[order[:left]] - torch.logsumexp(x, 0)
        bound = (vocab / 8192 + 64) * U + 2.0 ** -22 * (2 * math.log(vocab) + 2 + (x.max() - x[order[:left]])) + 2 * U * want.abs()
        assert ((got.top_logprobs[r, :left].double() - want).abs() <= bound).all(), r


# --------------------------------------------------------------------- norm --
def ref_norm(v, kind, w, b, eps, delta):
    """v in 64 bits with errors of at most delta: the norm and its bound of error."""
    if kind == 0:
        return v, delta
    N = v.shape[1]
    size = np.abs(v).mean(1, keepdims=True)
    if kind == 2:
        mean = v.mean(1, keepdims=True)
        delta = delta + delta.mean(1, keepdims=True) + 43 * U * size + U * np.abs(v)
        v = v - mean
    inv = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    # relative error of 1 / sqrt: the row's error beside its size, 42 / 2 + 4 roundings; no more than what eps leaves
    rel = np.sqrt((delta * delta).mean(1, keepdims=True)) * inv + 25 * U
    z = v * inv * w
    d = np.abs(w) * inv * delta + np.abs(z) * (rel + 3 * U)
    return z + b, d + U * (np.abs(z) + np.abs(z + b))


def rounded(d, exact, dtype):
    return d + (np.maximum(2.0 ** -11 * (np.abs(exact) + d), 2.0 ** -25) if dtype == torch.float16 else U * np.abs(exact))


NORMS = [
    # tokens, hidden, y, residual, gate, post, pre, bias
    (1, 1, "f32", "f32", "none", 0, 1, False), (3, 5, "f16", "f16", "channel", 1, 1, True), (1, 5120, "f32", "f32", "none", 0, 1, False),
    (13, 5003, "f16", "f16", "channel", 1, 1, False), (2, 64, "f32", "f16", "token", 2, 2, True), (9, 1000, "f16", "f32", "token", 1, 2, False),
    (400, 1028, "f32", "f32", "none", 1, 1, False), (5, 1023, "f32", "f32", "none", 2, 1, True), (170, 6144, "f16", "f32", "token", 2, 2, True),
    (2, 16388, "f32", "f32", "channel", 1, 1, False), (2, 32768, "f16", "f16", "none", 2, 2, False), (3, 32767, "f32", "f32", "token", 1, 2, True),
    (6, 640, None, "f32", "none", 0, 1, False), (6, 641, None, "f16", "none", 0, 2, True), (4, 256, "f32", None, "channel", 1, 1, False),
    (4, 4100, "f16", None, "none", 0, 0, False), (200, 2049, "f16", "f16", "none", 0, 2, False), (1, 20000, "f32", "f32", "token", 2, 1, True),
    (160, 6148, "f32", "f32", "none", 2, 1, True), (160, 6148, "f16", "f16", "token", 1, 2, False), (155, 16384, "f16", "f16", "none", 2, 1, False),
    (155, 16388, "f16", "f16", "channel", 1, 1, True), (160, 20480, "f16", "f32", "none", 2, 2, False), (160, 20484, "f32", "f16", "none", 1, 0, False),
    (155, 32768, "f32", "f32", "none", 0, 2, False), (155, 8195, "f16", "f16", "none", 1, 1, False), (155, 16385, "f32", "f32", "token", 2, 1, True),
    (155, 20483, "f16", "f32", "none", 0, 1, False), (3, 12288, "f32", "f32", "none", 2, 2, False), (300, 128, "f16", "f16", "none", 1, 2, True),
    (77, 132, "f32", "f32", "token", 2, 1, False), (300, 256, "f32", "f16", "none", 0, 1, False), (33, 516, "f16", "f32", "channel", 1, 1, True),
]


@pytest.mark.parametrize("tokens,hidden,y,residual,gate,post,pre,bias", NORMS)
def test_norm(pn, tokens, hidden, y, residual, gate, post, pre, bias):
    types = {"f32": torch.float32, "f16": torch.float16}
    g = torch.Generator().manual_seed(tokens + hidden)
    rand = lambda *s: torch.randn(*s, generator=g)
    Y = None if y is None else (2 * rand(tokens, hidden) + 3).to(types[y])        # a mean that is not small
    R = None if residual is None else (rand(tokens, hidden) * 5).to(types[residual])
    G = {"none": None, "channel": rand(hidden), "token": rand(tokens, hidden)}[gate]
    pw, pb = (1 + 0.2 * rand(hidden) if post else None), (rand(hidden) if post and bias else None)
    w, b = (1 + 0.2 * rand(hidden) if pre else None), (rand(hidden) if pre and bias else None)
    dev = lambda t: None if t is None else t.cuda()
    scale, eps = 0.37, 1e-5
    args = dict(gate=dev(G), scale=scale, post=post, post_weight=dev(pw), post_bias=dev(pb), pre=pre, pre_weight=dev(w), pre_bias=dev(b), eps=eps)
    r_got, x_got = pn.norm(dev(Y), dev(R), **args)
    num = lambda t, other=0.0: other if t is None else t.double().numpy()
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    zero = np.zeros((tokens, hidden))
    if y is None:
        r, d = num(R), zero
    else:
        z, d = ref_norm(num(Y), post, num(pw, 1.0), num(pb), eps, zero)
        f = scale * num(G, 1.0)
        r = num(R) + f * z
        d = np.abs(f) * d + 2 * U * np.abs(f * z) + U * np.abs(r)
    out_type = types[residual] if residual else torch.float32
    if y is None:
        assert r_got is None
    else:
        assert r_got.dtype == out_type
        limit = rounded(d, r, out_type)
        assert np.all(np.abs(num(r_got.cpu()) - r) <= limit), (np.abs(num(r_got.cpu()) - r) / limit).max()
    x, d = ref_norm(r, pre, num(w, 1.0), num(b), eps, d)
    limit = rounded(d, x, torch.float16)
    assert x_got.dtype == torch.float16
    assert np.all(np.abs(num(x_got.cpu()) - x) <= limit), (np.abs(num(x_got.cpu()) - x) / limit).max()
    # in place, and each output alone
    if y is not None and residual is not None:
        mine = dev(R)
        r2, x2 = pn.norm(dev(Y), mine, residual_out=mine, **args)
        assert r2 is mine and torch.equal(mine, r_got) and torch.equal(x2, x_got)
    if y is not None:
        only, none = pn.norm(dev(Y), dev(R), want_x=False, **args)
        assert none is None and torch.equal(only, r_got)
        none, only = pn.norm(dev(Y), dev(R), want_residual=False, **args)
        assert none is None and torch.equal(only, x_got)


@pytest.mark.parametrize("hidden", [100, 2048, 2051])
def test_norm_strides(pn, hidden):
    """Inputs and outputs that are columns of wider rows, at odd places too; nothing beside them is written."""
    T = 5
    g = torch.Generator(device="cuda").manual_seed(hidden)
    for shift in (0, 1, 4):
        wide = torch.randn(T, 2 * hidden + 16, generator=g, device="cuda")
        y, r = wide[:, shift:shift + hidden], torch.randn(T, hidden + 8, generator=g, device="cuda").half()[:, shift:shift + hidden]
        gate = torch.randn(T, hidden + 9, generator=g, device="cuda")[:, :hidden]
        out = torch.full((T, hidden + 12), 7.0, dtype=torch.float16, device="cuda")
        place = out[:, shift:shift + hidden]
        got, x = pn.norm(y, r, gate, residual_out=place)
        want, x_want = pn.norm(y.contiguous(), r.contiguous(), gate.contiguous())
        assert got is place
        # (fours and single values are added in another order)
        assert torch.equal(place, want) and (x.float() - x_want.float()).abs().max() <= 2.0 ** -9 * x_want.float().abs().max()
        out[:, shift:shift + hidden] = 7
        assert bool((out == 7).all())


def test_norm_large_mean_and_zero_rows(pn):
    """A mean 10^4 times the spread keeps its bits; rows of zeros give the bias."""
    N = 4096
    v = torch.randn(3, N, generator=torch.Generator().manual_seed(0)) + 1e4
    v[1] = 0
    b = torch.arange(N) / 64.0
    x = pn.norm(None, v.cuda(), pre=pn.NORM_LAYER, pre_bias=b.cuda(), eps=1e-6)[1].cpu().double()
    d = v.double()
    want = (d - d.mean(1, keepdim=True)) / (d.var(1, correction=0, keepdim=True) + 1e-6).sqrt() + b.double()
    # the mean errs by 43 u |v|, which is 0.026 here, beside a spread of 1: that moves all values alike
    assert (x[0] - want[0]).abs().max() <= 43 * U * 1.0005e4 + 2.0 ** -11 * want[0].abs().max() + 1e-3
    assert torch.equal(x[1], b.half().double())


# -------------------------------------------------------------------- weigh --
def weigh_case(lens, counts, heads, kv, D, page, seed=0):
    from test_gpu_serving import attention_case
    q, cache, table, lens, starts, ks, vs = attention_case(lens, counts, heads, kv, D, page, seed)
    rng = np.random.default_rng(seed + 1)
    weights = rng.random((cache.shape[0], kv, page)).astype(np.float32)
    return q, cache, table, lens, starts, ks, vs, weights


def check_weigh(pn, case, max_queries, scale, window=0, sinks=0, decay=1.0, with_weights=True, hidden=()):
    q, cache, table, lens, starts, ks, vs, weights = case
    dev = [cuda(a) for a in (q, cache, table, lens, starts)]
    page, group = cache.shape[2] * 16, q.shape[1] // cache.shape[1]
    _, lse = pn.attention(*dev, max_queries, scale, window=window, sinks=sinks, return_lse=True)
    before = cuda(weights) if with_weights else None
    out = torch.full(weights.shape, -3.0, device="cuda")
    got = pn.kv_weigh(*dev, max_queries, lse, scale, weights=before, decay=decay, out=out, window=window, sinks=sinks)
    assert got is out
    if with_weights:                                         # in place, the same bits where anything is written
        assert pn.kv_weigh(*dev, max_queries, lse, scale, weights=before, decay=decay, window=window, sinks=sinks) is before
        changed = out != -3
        assert torch.equal(before[changed], out[changed]) and torch.equal(before[~changed], cuda(weights)[~changed])
    got, lse = got.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    scale, decay = float(np.float32(scale)), float(np.float32(decay))
    written = np.zeros(got.shape, bool)
    for b in range(len(lens)):
        n, L = int(starts[b + 1] - starts[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        t = np.arange(L)
        total, bound = np.zeros((L, cache.shape[1])), np.zeros((L, cache.shape[1]))
        for i in range(n):
            p = L - n + i
            see = t <= p
            if window:
                see &= (t > p - window) | (t < sinks)
            see &= ~np.isin(t, [x for bb, x in hidden if bb == b])
            if not see.any():
                continue
            for h in range(q.shape[1]):
                k, row, z = ks[b][see, h // group], q[starts[b] + i, h].astype(np.float64), lse[starts[b] + i, h]
                x = scale * (k @ row)
                e = 2.0 ** -19 * abs(scale) * (np.abs(k) @ np.abs(row)) + 2.0 ** -22 * (np.abs(x) + abs(z) + 2) + 2.0 ** -21
                total[see, h // group] += np.exp(x - z)
                bound[see, h // group] += np.exp(x - z) * np.expm1(e)
        bound += total * (n * group / 4 + 12) * U
        slots = table[b, t // page].astype(np.int64) * page + t % page
        real = (slots >= 0) & (slots < cache.shape[0] * page)
        for h in range(cache.shape[1]):
            at = slots[real] // page, h, slots[real] % page
            old = np.where(t < L - n, decay * weights[at[0], h, at[2]] if with_weights else 0.0, 0.0) if real.all() else \
                np.where(t[real] < L - n, decay * weights[at[0], h, at[2]] if with_weights else 0.0, 0.0)
            want = old + total[real, h]
            limit = bound[real, h] + 2 * U * (old + want) + 1e-37
            assert np.all(np.abs(got[at] - want) <= limit), f"request {b}: {(np.abs(got[at] - want) / limit).max()}"
            written[at] = True
    assert np.all(got[~written] == -3)
    return got


WEIGHTS = [
    # lens, queries of each, heads, kv heads, D, page, window, sinks
    ([1], [1], 1, 1, 64, 16, 0, 0), ([1], [1], 8, 1, 128, 16, 0, 0), ([1], [1], 6, 1, 256, 16, 0, 0),
    ([15, 16, 17], [1, 1, 1], 4, 2, 128, 16, 0, 0), ([63, 64, 65, 0, 130], [1, 1, 1, 1, 1], 8, 2, 64, 32, 0, 0),
    ([200, 1, 77], [1, 1, 1], 10, 2, 256, 64, 0, 0), ([1000], [1], 16, 4, 128, 128, 0, 0), ([257, 511, 513], [1, 1, 0], 24, 1, 128, 32, 0, 0),
    ([40, 3, 64, 9], [4, 3, 0, 4], 4, 2, 128, 16, 0, 0), ([100, 2], [8, 8], 6, 1, 128, 32, 0, 0), ([333, 90], [7, 5], 12, 2, 64, 16, 0, 0),
    ([129, 500], [3, 16], 10, 2, 256, 16, 0, 0), ([500, 20, 64], [1, 1, 1], 4, 1, 128, 16, 100, 4), ([700], [1], 4, 4, 64, 64, 1, 0),
    ([700], [1], 8, 2, 256, 32, 64, 70), ([900, 350], [8, 3], 12, 2, 128, 16, 130, 17), ([300], [5], 2, 1, 128, 16, 1, 1),
    ([70], [70], 4, 2, 128, 16, 0, 0), ([200, 150], [130, 150], 6, 2, 64, 32, 0, 0), ([290], [257], 5, 1, 256, 64, 0, 0),
    ([400], [300], 4, 1, 128, 16, 90, 5), ([333, 40, 129], [200, 40, 1], 8, 1, 128, 64, 0, 0), ([130], [130], 3, 3, 256, 128, 33, 70),
    ([270], [270], 2, 2, 64, 16, 64, 0), ([600], [140], 8, 1, 128, 32, 0, 0), ([300], [40], 5, 1, 128, 64, 0, 0), ([700, 0, 5, 257], [64, 0, 5, 200], 6, 2, 256, 16, 0, 0),
    ([300, 128], [90, 127], 14, 2, 64, 16, 50, 9), ([200], [3], 130, 1, 128, 16, 0, 0), ([150], [4], 65, 1, 256, 16, 0, 0), ([129], [2], 128, 1, 128, 32, 0, 0),
    ([1500, 40], [1, 33], 8, 1, 128, 64, 0, 0),
    # rows to a key/value head: 17, 24, 28, 36, 44, 60, 64, 65, 90, 96, 97; 9, 17, 30, 32, 33; 200
    ([100, 517], [17, 9], 2, 2, 64, 16, 0, 0), ([300, 40, 7], [6, 1, 4], 8, 2, 128, 16, 0, 0), ([400, 65, 0, 33], [7, 7, 0, 7], 8, 2, 64, 32, 64, 3),
    ([290, 31], [9, 2], 12, 3, 128, 64, 100, 20), ([700], [11], 4, 1, 128, 16, 1, 0), ([129, 600], [15, 15], 4, 1, 64, 16, 0, 0),
    ([1000, 64], [16, 16], 8, 2, 128, 128, 0, 0), ([200], [13], 5, 1, 128, 32, 0, 0), ([333, 90, 91], [30, 1, 30], 3, 1, 64, 64, 30, 40),
    ([96, 500], [96, 40], 2, 2, 64, 16, 0, 0), ([97, 3], [97, 3], 1, 1, 64, 16, 0, 0), ([160, 20], [9, 2], 2, 2, 256, 16, 0, 0),
    ([300, 17, 1], [17, 17, 1], 1, 1, 256, 32, 0, 0), ([500, 200], [6, 3], 10, 2, 256, 64, 50, 6), ([400], [8], 4, 1, 256, 16, 0, 0),
    ([333, 32], [11, 4], 6, 2, 256, 16, 0, 0), ([77], [1], 200, 1, 64, 16, 0, 0), ([90, 300], [2, 1], 300, 2, 64, 32, 70, 2),
]


@pytest.mark.parametrize("lens,counts,heads,kv,D,page,window,sinks", WEIGHTS)
def test_weigh(pn, lens, counts, heads, kv, D, page, window, sinks):
    case = weigh_case(lens, counts, heads, kv, D, page)
    most = max(max(counts), 1)
    first = check_weigh(pn, case, most, 1 / math.sqrt(D), window, sinks)
    assert np.array_equal(first, check_weigh(pn, case, most, 1 / math.sqrt(D), window, sinks))
    check_weigh(pn, case, most, 1 / math.sqrt(D), window, sinks, decay=0.9)
    check_weigh(pn, case, most, 1 / math.sqrt(D), window, sinks, with_weights=False)


@pytest.mark.parametrize("counts", [[1, 1], [9, 20], [60, 33]])
@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0])
def test_weigh_sharp_and_flat(pn, counts, scale):
    check_weigh(pn, weigh_case([150, 33], counts, 4, 2, 128, 16, 1), max(counts), scale)


@pytest.mark.parametrize("counts", [[1, 1], [40, 40]])
def test_weigh_hidden_pages(pn, counts):
    """Tokens on pages outside the cache have no weight and no place; what a later token's scale holds reaches no earlier query."""
    case = list(weigh_case([100, 60], counts, 4, 1, 128, 16))
    table, cache = case[2], case[1]
    table[0, 1], table[0, 4] = -3, cache.shape[0]
    check_weigh(pn, case, max(counts), 0.1, hidden=[(0, t) for t in range(100) if t // 16 in (1, 4)])


def test_weigh_sums_to_the_rows(pn):
    """Over the tokens the weights of one step add up to the rows that see any; requests of a batch do not change one another's bits."""
    case = weigh_case([3000, 700, 1, 90], [1, 5, 1, 40], 8, 2, 128, 64, 3)
    q, cache, table, lens, starts, ks, vs, weights = case
    dev = [cuda(a) for a in (q, cache, table, lens, starts)]
    _, lse = pn.attention(*dev, 40, 0.09, return_lse=True)
    all_of = pn.kv_weigh(*dev, 40, lse, 0.09)
    assert all_of.shape == weights.shape
    total = all_of.double().sum((0, 2)).cpu()
    assert torch.all((total - 47 * 4).abs() <= 47 * 4 * 2.0 ** -14)
    for b in range(4):
        rows = slice(int(starts[b]), int(starts[b + 1]))
        one = pn.kv_weigh(dev[0][rows], dev[1], dev[2][b:b + 1], dev[3][b:b + 1], cuda(starts[b:b + 2] - starts[b]), 40, lse[rows], 0.09)
        pages = table[b, :-(-int(lens[b]) // 64)]
        assert torch.equal(one[pages], all_of[pages])


def test_weigh_long(pn):
    """One request over the whole GPU: its cache is one page's tokens over and over, so the weights repeat too."""
    D, kv, heads, page, L = 128, 2, 8, 64, 200001
    rng = np.random.default_rng(3)
    k = rng.standard_normal((page, kv, D)).astype(np.float32)
    kn, kd = ref.quantise(k)
    cache = np.full((1, kv, page // 16, 17 * D), 0x11, np.uint8)
    ref.write_tokens(cache, list(range(page)), kn, kd, kn, kd)
    kf = ref.dequantise(kn, kd)
    q = rng.standard_normal((1, heads, D)).astype(np.float16)
    table = np.zeros((1, -(-L // page)), np.int32)
    lse = rng.standard_normal((1, heads)).astype(np.float32) + 5
    got = pn.kv_weigh(cuda(q), cuda(cache), cuda(table), cuda(np.array([L], np.int32)), cuda(np.array([0, 1], np.int32)), 1, cuda(lse), 0.05).cpu().numpy()
    for h in range(kv):
        x = np.stack([0.05 * (kf[:, h] @ q[0, i].astype(np.float64)) - lse[0, i] for i in range(4 * h, 4 * h + 4)])
        assert np.abs(got[0, h] / np.exp(x).sum(0) - 1).max() <= 2.0 ** -15


WAYS = [(4, 2, 64, [1, 1]), (4, 2, 128, [1, 5]), (6, 2, 256, [7, 2]), (4, 2, 128, [70, 33]), (8, 1, 256, [9, 64]), (150, 1, 64, [2, 1])]


@pytest.mark.parametrize("heads,kv,D,counts", WAYS)
def test_weigh_strides(pn, heads, kv, D, counts):
    """Queries inside wider rows, tables that are part of wider ones, requests that others pad: the same bits."""
    case = weigh_case([200, 90], counts, heads, kv, D, 16, 4)
    q, cache, table, lens, starts = (cuda(a) for a in case[:5])
    lse = torch.randn(q.shape[0], heads, device="cuda") + 9
    want = pn.kv_weigh(q, cache, table, lens, starts, max(counts), lse, 0.1)
    wide_q = torch.full((q.shape[0], heads + 2 * kv, D), float("nan"), dtype=torch.float16, device="cuda")
    wide_q[:, :heads] = q
    wide_table = torch.full((2, table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    wide_table[:, 2:-3] = table
    got = pn.kv_weigh(wide_q[:, :heads], cache, wide_table[:, 2:-3], lens, starts, max(counts), lse, 0.1)
    assert torch.equal(got, want)
    # before, between and behind them requests of no queries or no tokens; tokens behind the last request
    pad = lambda t, v: torch.tensor([v[0], int(t[0]), v[1], int(t[1]), v[2]], dtype=torch.int32, device="cuda")  # noqa: E731
    more = torch.cat([table[:1], table[:1], table[:1], table[1:], table[1:]])
    n0, n = counts[0], sum(counts)
    begins = torch.tensor([0, 0, n0, n0, n, n], dtype=torch.int32, device="cuda")
    tail = torch.cat([q, torch.full_like(q[:1], float("inf"))])
    got = pn.kv_weigh(tail, cache, more, pad(lens, [150, 0, 17]), begins, max(counts), torch.cat([lse, lse[:1]]), 0.1)
    assert torch.equal(got, want)


@pytest.mark.parametrize("heads,kv,D,counts", WAYS)
def test_weigh_two_at_once(pn, heads, kv, D, counts):
    """Calls on two streams that overlap, and a captured one beside an eager one, do not disturb each other."""
    states = []
    for seed in (1, 2):
        case = weigh_case([3000, 900], counts, heads, kv, D, 16, seed)
        dev = [cuda(a) for a in case[:5]]
        lse = torch.randn(dev[0].shape[0], heads, device="cuda") + 9
        states.append((dev, lse, pn.kv_weigh(*dev, max(counts), lse, 0.1)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros_like(states[i][2]) for _ in range(5)] for i in range(2)]
    torch.cuda.synchronize()
    for k in range(5):
        for i, (dev, lse, _) in enumerate(states):
            pn.kv_weigh(*dev, max(counts), lse, 0.1, out=outs[i][k], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, states[i][2]) for i in range(2) for o in outs[i])
    graph = torch.cuda.CUDAGraph()
    dev, lse, want = states[0]
    with torch.cuda.graph(graph):
        got = pn.kv_weigh(*dev, max(counts), lse, 0.1)
    got.zero_()
    outs[1][0].zero_()
    torch.cuda.synchronize()
    graph.replay()
    pn.kv_weigh(*states[1][0], max(counts), states[1][1], 0.1, out=outs[1][0], stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(outs[1][0], states[1][2])


def test_weigh_wait_timeout(pn):
    """A wait on the GPU that gives up leaves NaN in the weights, and the next call is right."""
    case = weigh_case([300, 200], [80, 100], 4, 2, 128, 16)
    q, cache, table, lens, starts, ks, vs, weights = case
    dev = [cuda(a) for a in (q, cache, table, lens, starts)]
    lse = torch.zeros(180, 4, device="cuda")
    pn.set_wait_timeout_ns(20_000_000)
    pn.set_test_stall(True)
    try:
        out = pn.kv_weigh(*dev, 100, lse, 0.1)
        torch.cuda.synchronize()
    finally:
        pn.set_test_stall(False)
        pn.set_wait_timeout_ns(1_000_000_000)
    assert torch.isnan(out[table[0, :300 // 16]]).all()
    check_weigh(pn, case, 100, 0.1)


# -------------------------------------------------------------------- evict --
def ref_evict(weights, table, lens, held, free, ring, page, limit, budget, sinks, recent):
    """Request by request; free is written like the call does."""
    F, each = len(free), -(-budget // page)
    head, tail = (int(x) for x in ring)
    pages, kv = weights.shape[:2]
    table_out, lens_out, held_out = table.copy(), lens.copy(), held.copy()
    kept = np.full((len(lens), kv, budget), -1, np.int32)
    taken = back = refused = 0
    give = []
    for b in range(len(lens)):
        L = min(max(int(lens[b]), 0), table.shape[1] * page)
        if L <= limit:
            continue
        if taken + each > tail - head:
            refused += 1
            continue
        t = np.arange(L)
        at = table[b, t // page]
        for h in range(kv):
            w = np.array([weights[p, h, i % page] if 0 <= p < pages else -np.inf for i, p in enumerate(at)], np.float64)
            w = np.where(np.isnan(w), -np.inf, w)
            inner = sorted(range(sinks, L - recent), key=lambda i: (-w[i], i))[:budget - sinks - recent]
            kept[b, h] = sorted([*range(sinks), *inner, *range(L - recent, L)])
        table_out[b] = -1
        table_out[b, :each] = [free[(head + taken + i) % F] for i in range(each)]
        give += [int(p) for p in table[b, :held[b]]]
        taken, back = taken + each, back + int(held[b])
        lens_out[b], held_out[b] = budget, each
    for i, p in enumerate(give):
        free[(tail + i) % F] = p
    return dict(table=table_out, lens=lens_out, held=held_out, ring=np.array([head + taken, tail + back]), kept=kept, refused=np.array([refused]))


def evict_case(lens, kv, D, page, budget, spare=None, seed=0):
    rng = np.random.default_rng(seed + len(lens) + D)
    held = [-(-n // page) + int(rng.integers(0, 2)) for n in lens]
    most = max(held) + 1
    spare = len(lens) * -(-budget // page) if spare is None else spare
    pages = sum(held) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), most), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    head = int(rng.integers(0, 3 * pages))
    free = np.full(pages, -5, np.int32)
    for i in range(spare):
        free[(head + i) % pages] = order[at + i]
    cache = rng.integers(0, 256, (pages, kv, page // 16, 17 * D)).astype(np.uint8)
    cache[..., 8 * D + 1:8 * D + D // 2:2] &= 0xBF           # finite scales: an exponent bit less
    cache[..., 16 * D + D // 2 + 1::2] &= 0xBF
    weights = rng.random((pages, kv, page)).astype(np.float32)
    return cache, weights, table, np.array(lens, np.int32), np.array(held, np.int32), free, np.array([head, head + spare], np.int64)


def check_evict(pn, case, limit, budget, sinks, recent):
    cache, weights, table, lens, held, free, ring = case
    page, pages, kv = cache.shape[2] * 16, cache.shape[0], cache.shape[1]
    d_cache, d_weights, d_free = cuda(cache), cuda(weights), cuda(free)
    args = (cuda(table), cuda(lens), cuda(held), d_free, cuda(ring), limit, budget, sinks, recent)
    got = pn.kv_evict(d_cache, d_weights, *args)
    after = free.copy()
    want = ref_evict(weights, table, lens, held, after, ring, page, limit, budget, sinks, recent)
    for name in got._fields:
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    assert np.array_equal(d_free.cpu().numpy(), after)
    # codes, scales and weights are the kept tokens'
    touched = np.zeros(pages, bool)
    for b in range(len(lens)):
        if want["kept"][b, 0, 0] < 0:
            continue
        t = np.arange(budget)
        new = want["table"][b, t // page].astype(np.int64) * page + t % page
        touched[want["table"][b, :-(-budget // page)]] = True
        k_new, v_new = (x.cpu().numpy() for x in pn.kv_read(d_cache, cuda(new)))
        w_new = d_weights.cpu().numpy()
        for h in range(kv):
            p = want["kept"][b, h]
            old = np.where((table[b, p // page] >= 0) & (table[b, p // page] < pages), table[b, p // page].astype(np.int64) * page + p % page, -1)
            k_old, v_old = (x.cpu().numpy() for x in pn.kv_read(cuda(cache), cuda(old)))
            assert np.array_equal(k_new[:, h], k_old[:, h]) and np.array_equal(v_new[:, h], v_old[:, h])
            w_old = np.where(old >= 0, weights[old // page, h, old % page], 0)
            assert np.array_equal(w_new[new // page, h, new % page], w_old, equal_nan=True)
    assert np.array_equal(d_cache.cpu().numpy()[~touched], cache[~touched])
    assert np.array_equal(d_weights.cpu().numpy()[~touched], weights[~touched], equal_nan=True)
    # nothing behind the budget in the last page
    if budget % page and touched.any():
        for b in range(len(lens)):
            last = want["table"][b, budget // page]
            if want["kept"][b, 0, 0] >= 0:
                assert np.array_equal(d_weights.cpu().numpy()[last][:, budget % page:], weights[last][:, budget % page:], equal_nan=True)
                tail = slice(-(-(budget % page) // 16), None)
                assert np.array_equal(d_cache.cpu().numpy()[last][:, tail], cache[last][:, tail])
    # again on the same inputs, into the same outputs
    again = pn.kv_evict(d_cache, d_weights, *args, out=got)
    assert again.kept is got.kept
    for name in got._fields:
        assert np.array_equal(getattr(again, name).cpu().numpy(), want[name]), name
    return want


EVICTIONS = [
    # lens, kv heads, D, page, limit, budget, first, last, spare pages (None: plenty)
    ([2], 1, 64, 16, 1, 1, 0, 0, None), ([17], 2, 128, 16, 16, 16, 0, 16, None), ([100, 3, 0, 64], 2, 64, 16, 40, 33, 4, 9, None),
    ([200, 500, 90], 1, 256, 32, 80, 47, 0, 8, None), ([1000], 4, 128, 64, 256, 200, 4, 32, None), ([300, 301, 302, 299], 2, 128, 16, 299, 299, 1, 0, None),
    ([700, 20, 650, 800], 1, 64, 128, 100, 100, 100, 0, None), ([90, 80, 70, 100], 2, 128, 16, 64, 40, 2, 2, 7), ([90, 80], 2, 128, 16, 64, 40, 2, 2, 0),
    ([5000], 1, 128, 16, 4999, 4999, 0, 1, None), ([60000], 1, 64, 1024, 50000, 3000, 4, 100, None), ([400] * 40, 1, 64, 16, 200, 64, 1, 5, 91),
]


@pytest.mark.parametrize("lens,kv,D,page,limit,budget,sinks,recent,spare", EVICTIONS)
def test_evict(pn, lens, kv, D, page, limit, budget, sinks, recent, spare):
    want = check_evict(pn, evict_case(lens, kv, D, page, budget, spare), limit, budget, sinks, recent)
    if spare is not None:
        assert int(want["refused"][0]) > 0


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "special", "tiny", "huge"])
def test_evict_weights(pn, kind):
    """Ties, negative weights, zeros of both signs, infinities and NaN, subnormal differences, one digit in common."""
    case = list(evict_case([700, 333], 2, 64, 16, 100, seed=5))
    rng = np.random.default_rng(1)
    w = case[1]
    if kind == "equal":
        w[:] = 0.5
    elif kind == "few":
        w[:] = rng.integers(0, 3, w.shape)
    elif kind == "signs":
        w[:] = rng.integers(-3, 4, w.shape) * np.where(rng.random(w.shape) < 0.5, 1.0, -1.0)
        w[w == 0] = np.where(rng.random((w == 0).sum()) < 0.5, 0.0, -0.0)
    elif kind == "special":
        w[rng.random(w.shape) < 0.3] = np.nan
        w[rng.random(w.shape) < 0.1] = np.inf
        w[rng.random(w.shape) < 0.4] = -np.inf
    elif kind == "tiny":
        w[:] = rng.integers(0, 2000, w.shape) * np.float32(1e-45)
    else:
        w[:] = np.float32(1e30) * (1 + np.float32(2.0 ** -23) * rng.integers(0, 900, w.shape))
    check_evict(pn, case, 200, 100, 3, 10)


@pytest.mark.parametrize("kind", ["random", "equal", "few", "close", "zeros"])
@pytest.mark.parametrize("lens,kv,page,limit,budget,sinks,recent", [
    ([4100], 1, 16, 4000, 300, 2, 5),                  # shares of few positions to a block
    ([9000, 2, 8190], 2, 64, 5000, 5000, 0, 0),
    ([33333, 16385], 1, 128, 16000, 1000, 16, 64),
    ([850000], 1, 1024, 800000, 2000, 4, 100),         # more than a block's keys
])
def test_evict_split(pn, lens, kv, page, limit, budget, sinks, recent, kind):
    """Few and long requests: several blocks share a request and head."""
    case = list(evict_case(lens, kv, 64, page, budget, seed=9))
    rng = np.random.default_rng(2)
    w = case[1]
    if kind == "equal":
        w[:] = 0.25
    elif kind == "few":
        w[:] = rng.integers(0, 5, w.shape)
    elif kind == "close":
        w[:] = 1 + np.float32(2.0 ** -23) * rng.integers(0, 3000, w.shape)
    elif kind == "zeros":                              # all that counts in one block's share
        w[:] = 0
        w[case[2][0, :4]] = rng.random((4, kv, page))
    check_evict(pn, case, limit, budget, sinks, recent)


def test_evict_pages_outside(pn):
    """Old pages outside the cache: their tokens come last and become zeros; new ones outside: nothing is written there."""
    case = list(evict_case([200, 180], 1, 128, 16, 150, seed=2))
    case[2][0, 3], case[2][0, 5], case[2][1, 0] = -1, 1 << 20, case[0].shape[0]
    check_evict(pn, case, 160, 150, 2, 4)


def test_evict_shared_pages(pn):
    """Requests with pages in common are cut back each for itself; what they share is only read."""
    case = list(evict_case([300, 280, 150], 2, 128, 16, 60, seed=8))
    case[2][1, :6] = case[2][2, :6] = case[2][0, :6]
    check_evict(pn, case, 100, 60, 4, 9)


def test_evict_at_once(pn):
    """Two caches on two streams."""
    states = []
    for seed in (1, 2):
        cache, weights, table, lens, held, free, ring = evict_case([9000, 300], 2, 64, 32, 200, seed=seed)
        dev = [cuda(a) for a in (cache, weights, table, lens, held, free, ring)]
        states.append((dev, torch.cuda.Stream()))
    wants = [pn.kv_evict(*dev, 250, 200, 3, 20) for dev, _ in states]
    torch.cuda.synchronize()
    for _ in range(4):
        gots = [pn.kv_evict(*dev, 250, 200, 3, 20, stream=stream) for dev, stream in states]
        torch.cuda.synchronize()
        for got, want in zip(gots, wants):
            assert all(torch.equal(getattr(got, n), getattr(want, n)) for n in got._fields)


def test_evict_large_batch(pn):
    case = evict_case([int(n) for n in np.random.default_rng(4).integers(0, 60, 1500)], 1, 64, 16, 20, spare=1000)
    check_evict(pn, case, 30, 20, 1, 3)


# ------------------------------------------------------------------ together --
def test_streams_and_graphs(pn):
    """Every call captured into a graph and replayed on new inputs, and on a stream of its own, gives the same bits."""
    case = weigh_case([300, 41], [1, 1], 4, 2, 64, 16, 7)
    q, cache, table, lens, starts, ks, vs, weights = (cuda(a) if isinstance(a, np.ndarray) else a for a in case)
    lse = torch.randn(2, 4, device="cuda") + 6
    logits, tokens = torch.randn(3, 5000, device="cuda"), torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    y, r = torch.randn(4, 640, device="cuda"), torch.randn(4, 640, device="cuda")
    idle = sorted(set(range(cache.shape[0])) - set(case[2][case[2] < cache.shape[0]].tolist()))
    free, ring = torch.tensor(idle + [0] * 98, dtype=torch.int32, device="cuda"), torch.tensor([0, 2], device="cuda")
    held = (lens + 15) // 16

    def calls(stream=None):
        w = pn.kv_weigh(q, cache, table, lens, starts, 1, lse, 0.1, weights=weights, out=out_w, stream=stream)
        e = pn.kv_evict(cache, spare_w, table, lens, held, free, ring, 100, 32, 1, 4, stream=stream)
        return [w, e.kept, e.table, *pn.logprobs(logits, tokens, top=5, stream=stream), *pn.norm(y, r, stream=stream)]

    out_w, spare_w = torch.zeros_like(weights), weights.clone()
    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out_w.zero_()
    side.wait_stream(torch.cuda.current_stream())
    mine = calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(mine, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(2):
        for t in got[1:]:
            t.zero_()
        out_w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    logits.neg_()
    y.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    fresh = calls()
    assert all(torch.equal(a, b) for a, b in zip(got, fresh)) and not torch.equal(got[3], want[3])


def test_refusals(pn):
    x, i32 = torch.zeros(3, 64, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: pn.logprobs(x.double()), lambda: pn.logprobs(x, i32.long()), lambda: pn.norm(x, x, gate=x.half()),
                 lambda: pn.norm(x, pre_weight=x[0].half()), lambda: pn.norm(x, x, residual_out=x.half()), lambda: pn.norm(None, None)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: pn.logprobs(x[0]), lambda: pn.logprobs(x.T), lambda: pn.logprobs(x, i32[:2]), lambda: pn.logprobs(x, top=33),
                 lambda: pn.logprobs(x, top=-1), lambda: pn.norm(x, x[:2]), lambda: pn.norm(x.T), lambda: pn.norm(x, gate=x[:2]),
                 lambda: pn.norm(x, pre_weight=x[0, :5]), lambda: pn.norm(x, x=torch.zeros(3, 63, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pn.logprobs(x, scale=0.0), lambda: pn.logprobs(x, scale=math.nan), lambda: pn.norm(x, eps=-1.0), lambda: pn.norm(x, post=5),
                 lambda: pn.norm(x, residual_out=x), lambda: pn.norm(torch.zeros(1, 40000, device="cuda"))):
        with pytest.raises(pn.PnError) as e:
            call()
        assert e.value.status == 1
    assert pn.logprobs(x[:0]).entropy.shape == (0,)
    r, v = pn.norm(x[:0], x[:0])
    assert r.shape == (0, 64) and v.shape == (0, 64)
    cache, table, ring = pn.kv_cache(4, 16, 2, 64), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.tensor([0, 0], device="cuda")
    weights, free = pn.kv_weights(cache), torch.zeros(4, dtype=torch.int32, device="cuda")
    assert weights.shape == (4, 2, 16)
    q, lse, starts = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda"), torch.zeros(3, 4, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pn.kv_weigh(q, cache, table, i32, starts, 1, lse, 0.1, out=weights[:3])
    with pytest.raises(ValueError):
        pn.kv_weigh(q, cache, table, i32, starts, 1, lse[:2], 0.1, out=weights)
    with pytest.raises(pn.PnError):
        pn.kv_weigh(q, cache, table, i32, starts, 1, lse, 0.1, weights=weights, decay=2.0)
    for limit, budget, sinks, recent in ((4, 5, 0, 0), (4, 0, 0, 0), (4, 4, 3, 2)):
        with pytest.raises(pn.PnError) as e:
            pn.kv_evict(cache, weights, table, i32, i32, free, ring, limit, budget, sinks, recent)
        assert e.value.status == 1
    ok = pn.kv_evict(cache, weights, table, i32, i32, free, ring, 4, 4)
    assert ok.refused.item() == 0 and bool((ok.kept == -1).all()) and torch.equal(ok.table, table)
    with pytest.raises(pn.PnError):                           # the state of a call may not be its output
        pn.kv_evict(cache, weights, ok.table, ok.lens, ok.held, free, ok.ring, 4, 4, out=ok)


def test_bounded_cache_steps(pn):
    """Steps of a batch whose requests are cut back again and again, against tokens, weights and attention kept in 64 bits:
    outputs of attention over what is kept, gathered weights, what is kept, and no page lost."""
    heads, kv, D, page, limit, budget, sinks, recent, scale = 4, 2, 64, 16, 40, 24, 2, 8, 0.2
    B, group = 3, 2
    g = torch.Generator(device="cuda").manual_seed(11)
    most = -(-64 // page) + 1
    F = B * (most + -(-budget // page))
    cache = pn.kv_cache(F, page, kv, D)
    weights = pn.kv_weights(cache)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, free, ring = torch.zeros(B, most, **i32), torch.arange(F, **i32), torch.tensor([0, F], device="cuda")
    lens, held, gone = (torch.zeros(B, **i32) for _ in range(3))
    ws = pn.AttentionWorkspace()
    # of each request and head: keys, values, weights and first positions of what is kept
    kept = [[dict(k=np.zeros((0, D)), v=np.zeros((0, D)), w=np.zeros(0), p=np.zeros(0, np.int64)) for _ in range(kv)] for _ in range(B)]
    total, evictions = np.zeros(B, np.int64), 0
    angle = torch.arange(200, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    for turn in range(50):
        counts = [30, 5, 50] if turn == 0 else [1, 1, 1] if turn % 7 else [1, 3, 2]
        T = sum(counts)
        q, k, v = (torch.randn(T, n, D, generator=g, device="cuda") for n in (heads, kv, kv))
        plan = pn.kv_plan(lens, torch.tensor(counts, **i32), held, table, free, ring, page, T)
        positions = plan.positions + gone[plan.requests.long()]
        assert positions.tolist() == [int(total[b]) + i for b in range(B) for i in range(counts[b])]
        q16 = pn.kv_append(q, k, v, cache, plan.slots, positions, angle.cos(), angle.sin())
        out, lse = pn.attention(q16, cache, table, plan.lens, plan.starts, 50, scale, workspace=ws, return_lse=True)
        pn.kv_weigh(q16, cache, table, plan.lens, plan.starts, 50, lse, scale, weights=weights)
        ks, vs = (x.cpu().numpy().astype(np.float64) for x in pn.kv_read(cache, plan.slots))
        qs, out = q16.cpu().numpy().astype(np.float64), out.cpu().numpy().astype(np.float64)
        table_host, w_host = table.cpu().numpy(), weights.cpu().numpy()
        row = 0
        for b in range(B):
            rows = slice(row, row + counts[b])
            row += counts[b]
            for h in range(kv):
                s = kept[b][h]
                s["k"], s["v"] = np.concatenate([s["k"], ks[rows, h]]), np.concatenate([s["v"], vs[rows, h]])
                s["w"], s["p"] = np.concatenate([s["w"], np.zeros(counts[b])]), np.concatenate([s["p"], total[b] + np.arange(counts[b])])
                L = len(s["w"])
                for i, r in enumerate(range(rows.start, rows.stop)):
                    see = np.arange(L) <= L - counts[b] + i
                    for j in range(group):
                        x = np.where(see, scale * (s["k"] @ qs[r, h * group + j]), -np.inf)
                        p = np.exp(x - x.max())
                        p /= p.sum()
                        s["w"] += p
                        # (attention's own bound with room: p d is rounded once, the output once)
                        assert np.all(np.abs(out[r, h * group + j] - p @ s["v"]) <= 2.0 ** -9 * (p @ np.abs(s["v"])) + 2.0 ** -24)
                t = np.arange(L)
                mine = w_host[table_host[b, t // page], h, t % page]
                assert np.all(np.abs(mine - s["w"]) <= 2.0 ** -14 * s["w"] + 1e-6)
            total[b] += counts[b]
        e = pn.kv_evict(cache, weights, table, plan.lens, plan.held, free, plan.ring, limit, budget, sinks, recent)
        assert e.refused.item() == 0
        chosen = e.kept.cpu().numpy()
        for b in range(B):
            if chosen[b, 0, 0] < 0:
                continue
            evictions += 1
            for h in range(kv):
                s, c = kept[b][h], chosen[b, h]
                L = len(s["w"])
                assert np.all(np.diff(c) > 0) and c[:sinks].tolist() == list(range(sinks)) and c[-recent:].tolist() == list(range(L - recent, L))
                inner, dropped = c[sinks:-recent], np.setdiff1d(np.arange(sinks, L - recent), c)
                if len(dropped):
                    assert s["w"][inner].min() >= s["w"][dropped].max() * (1 - 2.0 ** -13) - 2e-6
                for name in s:
                    s[name] = s[name][c]
        gone = gone + plan.lens - e.lens
        table, lens, held, ring = e.table, e.lens, e.held, e.ring
        h_host = held.tolist()
        mine = [p for b in range(B) for p in table.cpu()[b, :h_host[b]].tolist()]
        head, tail = ring.tolist()
        assert sorted(mine + [int(free[i % F]) for i in range(head, tail)]) == list(range(F))
        assert lens.tolist() == [len(kept[b][0]["w"]) for b in range(B)]
    assert evictions >= 8 and ws.status() == 0


def test_bounded_cache_example(pn):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import bounded_cache as e
    model = e.Model()
    prompts = [[7, 8, 9, 7, 8], list(range(100, 163)), [3]]
    whole, logprobs, pages = e.generate(model, prompts, 50, 4096, 4096)
    assert all(len(t) == 50 and all(0 <= x < e.VOCAB for x in t) for t in whole)
    assert bool((logprobs <= 0).all()) and pages == -(-(63 + 49) // e.PAGE)
    # a limit that nothing reaches changes nothing; one that is reached bounds the pages
    again, same, _ = e.generate(model, prompts, 50, 200, 100)
    assert again == whole and torch.equal(same, logprobs)
    cut, _, pages = e.generate(model, prompts, 50, 64, 48)
    assert all(len(t) == 50 for t in cut) and pages <= -(-65 // e.PAGE)
