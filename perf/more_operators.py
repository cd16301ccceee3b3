"""Measured cases of the operators around a decoding step with a bounded cache.

Between the GEMVs, the cache and the answer of a decoding step stand

  norm      a block's output into the residual stream, with the norms before and after it,
            its gate and its scale, and the next GEMV's fp16 input (pn.norm)
  logprobs  log probabilities of given tokens, the entropy and the top alternatives from
            the vocabulary GEMV's logits (pn.logprobs)
  weigh     the attention weight that each cached token has gathered from the step's
            queries, added to what it had (pn.kv_weigh)
  evict     requests past a limit keep, for each head, first and last tokens and those of
            the largest weight, moved into fresh pages (pn.kv_evict; pn.kv_read reads them)

``run`` computes an operator in plain torch operations (``own`` false) or through
the framework's entry points (``own`` true); ``exact`` restates it in 64 bits.

The cache is the 4-bit one: uint8 [pages][kv_heads][page_size / 16][17 D], a record of 16
tokens of one head: K codes (8 D bytes), K scales (D / 2), V codes (8 D), V scales (D / 2);
values d (n - 8) in groups of 64 with an fp16 scale d, eight codes to a 32-bit word (code c
in half c & 1, at bit 4 (c >> 1)).  With h = token / 8, groups two by two in planes (one to
a plane for D = 64), and word i of a group, the words lie in the order
  K  [h][plane][token % 8][i / 2][group in plane][i % 2]
  V  [h][plane][i][token % 8 / 2][token % 2][group in plane]
and the scales [token][group].  Weights: fp32 [pages][kv_heads][page_size].
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one token between two GEMVs of the 27B-class layer: latency
        dict(name="norm_1", op="norm", tokens=1, hidden=5120, y="f32", residual="f32", gate="none", post="none", pre="rms", bias=False, scale=1.0),
        # a verification batch with norms before and after the block, a gate for each channel, rows of odd length
        dict(name="norm_verify_13", op="norm", tokens=13, hidden=5003, y="f16", residual="f16", gate="channel", post="rms", pre="rms", bias=False, scale=0.22),
        # a prompt chunk's residual stream in fp32: bound by memory
        dict(name="norm_prompt_8192", op="norm", tokens=8192, hidden=5120, y="f32", residual="f32", gate="none", post="none", pre="rms", bias=False, scale=1.0),
        # a block modulated token by token, mean and variance norms with biases
        dict(name="norm_gated_4096", op="norm", tokens=4096, hidden=6144, y="f16", residual="f32", gate="token", post="layer", pre="layer", bias=True, scale=0.5),
        # the token just drawn, with five alternatives, a small vocabulary: latency
        dict(name="logprobs_1", op="logprobs", rows=1, vocab=32000, dtype="f32", count=1, top=5, masked=0.0, scale=1.0),
        # a decode batch that asks for twenty alternatives
        dict(name="logprobs_64", op="logprobs", rows=64, vocab=151936, dtype="f32", count=1, top=20, masked=0.0, scale=1.0 / 0.7),
        # a prompt scored token by token, from half-precision logits
        dict(name="logprobs_prompt_2000", op="logprobs", rows=2000, vocab=151936, dtype="f16", count=1, top=1, masked=0.0, scale=1.0),
        # one very long request's decode step
        dict(name="weigh_1_long", op="weigh", batch=1, longest=131072, shortest=131072, queries=1, heads=48, kv_heads=8, dim=128, page=64, window=0, sinks=0, decay=1.0),
        # a decode batch of ragged lengths, older weight fading
        dict(name="weigh_64_ragged", op="weigh", batch=64, longest=16384, shortest=1, queries=1, heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0, decay=0.99),
        # a prompt chunk's queries over what is cached of it, heads of 256
        dict(name="weigh_prompt_2048", op="weigh", batch=1, longest=8192, shortest=8192, queries=2048, heads=24, kv_heads=4, dim=256, page=16, window=0, sinks=0, decay=0.0),
        # one conversation that has passed its limit: latency
        dict(name="evict_1", op="evict", batch=1, longest=1281, shortest=1281, kv_heads=4, dim=256, page=16, limit=1280, budget=1024, sinks=4, recent=64, spare=1.0),
        # a batch whose long requests are cut back to 512 tokens
        dict(name="evict_64", op="evict", batch=64, longest=16384, shortest=1, kv_heads=8, dim=128, page=64, limit=1024, budget=512, sinks=4, recent=128, spare=1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "logprobs", "logprobs", "weigh", "weigh", "evict"])
    if op == "norm":
        hidden = _log(rng, 64, 20000)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        return dict(op=op, tokens=_log(rng, 1, max(2, min(16384, 8192 * 5120 // hidden // 2))), hidden=hidden, y=rng.choice(["f32", "f16"]),
                    residual=rng.choice(["f32", "f16"]), gate=rng.choice(["none", "none", "channel", "token"]), post=rng.choice(["none", "rms", "layer"]),
                    pre=rng.choice(["rms", "rms", "layer"]), bias=rng.random() < 0.3, scale=rng.choice([1.0, 0.22, 1.5]))
    if op == "logprobs":
        vocab = _log(rng, 100, 200000)
        return dict(op=op, rows=_log(rng, 1, max(2, 2000 * 151936 // vocab // 4)) if vocab > 5000 else _log(rng, 1, 4000), vocab=vocab,
                    dtype=rng.choice(["f32", "f16"]), count=rng.choice([1, 1, 3]), top=rng.choice([0, 1, 5, 20, 32]), masked=rng.choice([0.0, 0.0, 0.7]),
                    scale=rng.choice([1.0, 0.5, 1.25]))
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    if op == "weigh":
        group = rng.choice([1, 2, 4, 5, 6, 8])
        kind = rng.choice(["one", "one", "drafts", "prompt"])
        queries = 1 if kind == "one" else rng.randint(2, 16) if kind == "drafts" else _log(rng, 17, 2048)
        batch = _log(rng, 1, 128) if kind != "prompt" else rng.randint(1, 4)
        # what the largest listed cases read and multiply
        most = min(131072, 64 * 16384 * 8 * 128 // (batch * kv * dim), 2048 * 24 * 256 * 7168 // (batch * queries * kv * group * dim))
        longest = max(queries, _log(rng, 1, max(2, most)))
        windowed = rng.random() < 0.3
        return dict(op=op, batch=batch, longest=longest, shortest=rng.choice([1, longest]), queries=queries, heads=kv * group, kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), window=_log(rng, 1, longest + 1) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0,
                    decay=rng.choice([0.0, 1.0, 0.9]))
    batch = _log(rng, 1, 64)
    page = rng.choice([16, 32, 64, 128])
    longest = _log(rng, 64, min(131072, 64 * 16384 * 8 * 128 // (batch * kv * dim)))
    limit = rng.randint(max(8, longest // 16), longest - 1)
    budget = rng.randint(max(1, limit // 4), limit)
    budget = min(budget, max(1, 64 * 512 * 8 * 128 // (batch * kv * dim)))
    sinks = rng.randint(0, min(budget // 4, 16))
    return dict(op=op, batch=batch, longest=longest, shortest=rng.choice([1, longest]), kv_heads=kv, dim=dim, page=page, limit=limit, budget=budget,
                sinks=sinks, recent=rng.randint(0, (budget - sinks) // 2), spare=rng.choice([1.0, 1.0, 0.6]))


# ----------------------------------------------------------------- inputs --
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


_TYPES = {"f32": torch.float32, "f16": torch.float16}


def prepare(case, seed):
    g = _generator(seed)
    return dict(case=case, **{"norm": _prepare_norm, "logprobs": _prepare_logprobs, "weigh": _prepare_weigh, "evict": _prepare_evict}[case["op"]](case, g))


def _randint(g, lo, hi, size):
    """Whole numbers from lo to hi, both included."""
    return torch.randint(lo, hi + 1, size, generator=g, device=DEV)


def _prepare_norm(c, g):
    T, N = c["tokens"], c["hidden"]
    loud = 0.5 + 2 * torch.rand(N, generator=g, device=DEV) ** 3                    # a few loud channels
    y = (loud * torch.randn(T, N, generator=g, device=DEV)).to(_TYPES[c["y"]])
    residual = (3 * loud * torch.randn(T, N, generator=g, device=DEV) + 0.3).to(_TYPES[c["residual"]])
    gate = None if c["gate"] == "none" else torch.randn(*((N,) if c["gate"] == "channel" else (T, N)), generator=g, device=DEV)
    s = dict(y=y, residual=residual, gate=gate)
    for at in ("post", "pre"):
        have = c[at] != "none"
        s[at + "_weight"] = 1 + 0.2 * torch.randn(N, generator=g, device=DEV) if have else None
        s[at + "_bias"] = 0.1 * torch.randn(N, generator=g, device=DEV) if have and c["bias"] else None
    return s


def _prepare_logprobs(c, g):
    R, V = c["rows"], c["vocab"]
    logits = torch.randn(R, V, generator=g, device=DEV)
    logits *= 2
    likely = _randint(g, 0, V - 1, (R, min(4, V)))                                  # tokens that the model leans to, more or less
    logits.scatter_add_(1, likely, 4 + 9 * torch.rand(likely.shape, generator=g, device=DEV))
    if c["masked"]:
        hide = torch.rand(R, V, generator=g, device=DEV) < c["masked"]              # a grammar's forbidden tokens
        logits.masked_fill_(hide.scatter(1, likely[:, :1], False), -math.inf)
    # given tokens: a likely one, then any (forbidden ones among them)
    tokens = torch.cat([likely[:, :1], _randint(g, 0, V - 1, (R, c["count"] - 1))], 1)
    return dict(logits=logits.to(_TYPES[c["dtype"]]), tokens=tokens.int())


def _cache_of(g, pages, KV, page, D):
    cache = torch.empty(pages, KV, page // 16, 17 * D, dtype=torch.uint8, device=DEV)
    loud = 0.5 + 2 * torch.rand(2, KV, D, generator=g, device=DEV) ** 3
    step = max(1, (1 << 26) // (KV * page * D))       # pages at a time, for the memory that quantising takes
    for at in range(0, pages, step):
        n = min(step, pages - at)
        k, v = (loud[i, None, :, None] * torch.randn(n, KV, page, D, generator=g, device=DEV) for i in range(2))
        cache[at:at + n] = _records(*_quantise(k), *_quantise(v))
    return cache


def _lengths(c, g):
    lens = _randint(g, c["shortest"], c["longest"], (c["batch"],))
    lens[0] = c["longest"]
    return lens


def _page_table(g, held, most, pages):
    """A table of requests' pages in any order, `most` to a request, and the pages that are left."""
    order = torch.randperm(pages, generator=g, device=DEV).int()
    used = int(held.sum())
    table = torch.zeros(len(held), most, dtype=torch.int32, device=DEV)
    table[torch.arange(most, device=DEV) < held[:, None]] = order[:used]
    return table, order[used:]


def _prepare_weigh(c, g):
    B, H, KV, D, page, nq = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["queries"]
    lens = _lengths(c, g)
    starts = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    starts[1:] = lens.clamp(max=nq).cumsum(0)         # a request shorter than the others' drafts has fewer queries
    held = (lens + page - 1) // page
    most = -(-c["longest"] // page)
    pages = B * most + 3
    table, _ = _page_table(g, held, most, pages)
    cache = _cache_of(g, pages, KV, page, D)
    q = torch.randn(int(starts[-1]), H, D, generator=g, device=DEV).half()
    weights = 2 * torch.rand(pages, KV, page, generator=g, device=DEV) ** 4
    s = dict(q=q, cache=cache, table=table, lens=lens.int(), starts=starts, scale=1.5 / math.sqrt(D), weights=weights, out=torch.zeros_like(weights))
    s["lse"] = _in_parts(dict(s, case=c), _log_sums)                    # as attention leaves them
    return s


def _prepare_evict(c, g):
    B, KV, D, page = c["batch"], c["kv_heads"], c["dim"], c["page"]
    lens = _lengths(c, g)
    # some requests hold a page more than they need
    held = (lens + page - 1) // page + (torch.rand(B, generator=g, device=DEV) < 0.2)
    each, most = -(-c["budget"] // page), -(-c["longest"] // page) + 1
    over = int((lens > c["limit"]).sum())
    spare = max(1, int(each * over * c["spare"]))
    pages = B * (most + each)
    table, rest = _page_table(g, held, most, pages)
    head = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
    free = torch.zeros(pages, dtype=torch.int32, device=DEV)
    free[(head + torch.arange(spare, device=DEV)) % pages] = rest[:spare]
    # weight gathered over many steps: a few tokens have most of it
    weights = torch.exp(1.5 * torch.randn(pages, KV, page, generator=g, device=DEV))
    t = torch.arange(c["budget"], device=DEV)
    new = rest[:min(over, spare // each) * each].long().reshape(-1, each)
    slots = torch.full((B, c["budget"]), -1, dtype=torch.int64, device=DEV)         # where the kept tokens will be
    slots[:len(new)] = new[:, t // page] * page + t % page
    return dict(cache=_cache_of(g, pages, KV, page, D), weights=weights, table=table, lens=lens.int(), held=held.int(), free=free,
                ring=torch.tensor([head, head + spare], dtype=torch.int64, device=DEV), slots=slots.flatten())


# -------------------------------------------------------- the 4-bit cache --
def _quantise(x):
    """fp32 [..., D] -> codes uint8 [..., D], scales fp16 [..., D / 64] (pn4t's signed-scale rule)."""
    x = x.unflatten(-1, (-1, 64))
    size = x.abs()
    top = size.amax(-1, keepdim=True)
    first = torch.where(size == top, torch.arange(64, device=x.device), 64).amin(-1, keepdim=True)
    d = (x.gather(-1, first) / -8.0).clamp(-65504.0, 65504.0).half()
    d = torch.where(d == 0, torch.zeros_like(d), d)
    n = torch.where(d == 0, 0.0, torch.round(x / d.float())).clamp(-8, 7) + 8
    return n.to(torch.uint8).flatten(-2), d.squeeze(-1)


def _planes(D):
    """(planes, groups to a plane)."""
    return max(1, D // 128), min(2, D // 64)


def _words(n):
    """codes [..., 8] -> 32-bit words [...]."""
    c = torch.arange(8, device=n.device)
    w = (n.to(torch.int64) << (16 * (c & 1) + 4 * (c >> 1))).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _records(kn, kd, vn, vd):
    """codes [pages][KV][page][D] and scales [pages][KV][page][D / 64] of K and V -> uint8 [pages][KV][page / 16][17 D]."""
    D = kn.shape[-1]
    planes, each = _planes(D)
    lead = kn.shape[:2] + (kn.shape[2] // 16,)

    def place(n, tokens, words, order):
        w = _words(n.unflatten(-1, (-1, 8)))                         # [pages][KV][page][D / 8]
        w = w.reshape(lead + tokens + (planes, each) + words)
        return w.permute(0, 1, 2, *(3 + i for i in order)).reshape(lead + (2 * D,)).view(torch.uint8)

    k = place(kn, (2, 8), (4, 2), (0, 2, 1, 4, 3, 5))                # h, token, plane, group, i / 2, i % 2
    v = place(vn, (2, 4, 2), (8,), (0, 3, 5, 1, 2, 4))               # h, token / 2, token % 2, plane, group, i
    scales = [d.contiguous().view(lead + (D // 4,)).view(torch.uint8) for d in (kd, vd)]
    return torch.cat([k, scales[0], v, scales[1]], -1)


def _token_bytes(D):
    """[16][17 D / 16]: the places in a record of each token's bytes: K codes, K scales, V codes, V scales."""
    planes, each = _planes(D)
    t = torch.arange(16, device=DEV)
    word = torch.arange(2 * D, device=DEV)
    k = word.reshape(2, planes, 8, 4, each, 2).permute(0, 2, 1, 4, 3, 5).reshape(16, D // 8)
    v = word.reshape(2, planes, 8, 4, 2, each).permute(0, 3, 4, 1, 5, 2).reshape(16, D // 8)
    in_word = torch.arange(4, device=DEV)
    codes = [(4 * w[..., None] + in_word).reshape(16, D // 2) for w in (k, v)]
    scales = t[:, None] * (D // 32) + torch.arange(D // 32, device=DEV)
    return torch.cat([codes[0], 8 * D + scales, 8 * D + D // 2 + codes[1], 16 * D + D // 2 + scales], -1)


def _token_values(c, cache, slots, which):
    """The keys (which = 0) or values (1) of `slots` [...] of every head: fp32 [..., KV, D]."""
    KV, D, page = c["kv_heads"], c["dim"], c["page"]
    at, r = slots // page, slots % page
    record = (at[..., None] * KV + torch.arange(KV, device=DEV)) * (page // 16) + (r // 16)[..., None]
    places = _token_bytes(D).chunk(2, 1)[which]
    data = cache.flatten()[record[..., None] * (17 * D) + places[r % 16][..., None, :]]
    words = data[..., :D // 2].contiguous().view(torch.int32)                       # group after group
    code = torch.arange(8, device=DEV, dtype=torch.int32)
    n = ((words[..., None] >> (16 * (code & 1) + 4 * (code >> 1))) & 15).flatten(-2).unflatten(-1, (-1, 64))
    d = data[..., D // 2:].contiguous().view(torch.float16).float()[..., None]
    return (d * (n - 8).float()).flatten(-2)


# -------------------------------------------------------------------- run --
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "logprobs": _own_logprobs, "weigh": _own_weigh, "evict": _own_evict}[op](state)
    return {"norm": _plain_norm, "logprobs": _plain_logprobs, "weigh": _plain_weigh, "evict": _plain_evict}[op](state)


def _own_norm(s):
    from bit_weight_only_pn_gb300 import pn
    kind = {"none": pn.NORM_NONE, "rms": pn.NORM_RMS, "layer": pn.NORM_LAYER}
    residual, x = pn.norm(s["y"], s["residual"], gate=s["gate"], scale=s["case"]["scale"], post=kind[s["case"]["post"]], post_weight=s["post_weight"],
                          post_bias=s["post_bias"], pre=kind[s["case"]["pre"]], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=1e-6)
    return dict(residual=residual, x=x)


def _own_logprobs(s):
    from bit_weight_only_pn_gb300 import pn
    p = pn.logprobs(s["logits"], s["tokens"], top=s["case"]["top"], scale=s["case"]["scale"])
    return dict(logprobs=p.logprobs, entropy=p.entropy, top_tokens=p.top_tokens, top_logprobs=p.top_logprobs)


def _own_weigh(s):
    from bit_weight_only_pn_gb300 import pn
    c = s["case"]
    return dict(weights=pn.kv_weigh(s["q"], s["cache"], s["table"], s["lens"], s["starts"], max_queries=c["queries"], lse=s["lse"], scale=s["scale"],
                                    weights=s["weights"], decay=c["decay"], out=s["out"], window=c["window"], sinks=c["sinks"]))


def _own_evict(s):
    from bit_weight_only_pn_gb300 import pn
    c = s["case"]
    e = pn.kv_evict(s["cache"], s["weights"], s["table"], s["lens"], s["held"], s["free"], s["ring"], limit=c["limit"], budget=c["budget"],
                    sinks=c["sinks"], recent=c["recent"])
    k, v = pn.kv_read(s["cache"], s["slots"])
    return dict(table=e.table, lens=e.lens, held=e.held, ring=e.ring, kept=e.kept, refused=e.refused, free=s["free"], weights=s["weights"], k=k, v=v)


def _normed(x, kind, weight, bias):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    return x if bias is None else x + bias


def _plain_norm(s):
    c = s["case"]
    y = _normed(s["y"].float(), c["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        y = y * s["gate"]
    r = s["residual"].float() + c["scale"] * y
    return dict(residual=r.to(s["residual"].dtype), x=_normed(r, c["pre"], s["pre_weight"], s["pre_bias"]).half())


def _plain_logprobs(s):
    c = s["case"]
    raw = s["logits"].float()
    x = raw * c["scale"]
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    d = x - top
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = (log_total - torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / total)[:, 0]
    index = torch.arange(c["vocab"], device=DEV, dtype=torch.int32)
    tokens, values = [], []
    left = raw
    for i in range(c["top"]):                         # the largest, the lowest index where several are, -1 where none is left
        most = left.amax(-1, keepdim=True)
        at = torch.where(left == most, index, c["vocab"]).amin(-1, keepdim=True)
        there = most > -math.inf
        tokens.append(torch.where(there, at, -1))
        values.append(torch.where(there, most * c["scale"] - top - log_total, -math.inf))
        left = left.scatter(1, at.long(), -math.inf)
    return dict(logprobs=d.gather(1, s["tokens"].long()) - log_total, entropy=entropy,
                top_tokens=torch.cat(tokens, 1) if tokens else None, top_logprobs=torch.cat(values, 1) if values else None)


def _visible(c, lens, counts, most_q, length):
    """[B][most_q][length]: which cached tokens a request's queries see; its last query sits at the last token."""
    at = (lens - counts)[:, None, None] + torch.arange(most_q, device=DEV)[None, :, None]
    t = torch.arange(length, device=DEV)[None, None, :]
    see = (t <= at) & (t < lens[:, None, None]) & (torch.arange(most_q, device=DEV) < counts[:, None])[:, :, None]
    return see & ((t > at - c["window"]) | (t < c["sinks"])) if c["window"] else see


def _in_parts(s, part):
    """part(s, b0, b1) over ranges of requests small enough for their scores, put together."""
    c = s["case"]
    each = max(1, (1 << 31) // max(1, c["queries"] * c["heads"] * c["longest"]))
    return torch.cat([part(s, b, min(b + each, c["batch"])) for b in range(0, c["batch"], each)])


def _scores(s, b0, b1):
    """Requests b0 .. b1 - 1: scores fp32 [B][KV][queries][group][L], -inf where hidden, rows of q [B][queries] and which are real."""
    c = s["case"]
    H, KV, D, nq, page = c["heads"], c["kv_heads"], c["dim"], c["queries"], c["page"]
    lens, starts = s["lens"][b0:b1].long(), s["starts"][b0:b1 + 1].long()
    counts = starts[1:] - starts[:-1]
    L = int(lens.max())
    table = s["table"][b0:b1].long()
    t = torch.arange(L, device=DEV)
    slots = torch.where(t < lens[:, None], table[:, t // page] * page + t % page, 0)
    k = _token_values(c, s["cache"], slots, 0).permute(0, 2, 1, 3)
    row = (starts[:-1, None] + torch.arange(nq, device=DEV)).clamp(max=len(s["q"]) - 1)
    q = s["q"].float()[row].reshape(b1 - b0, nq, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(b1 - b0, KV, -1, D)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).reshape(b1 - b0, KV, nq, H // KV, L)
    x.masked_fill_(~_visible(c, lens, counts, nq, L)[:, None, :, None, :], -math.inf)
    return x, row, torch.arange(nq, device=DEV) < counts[:, None]


def _log_sums(s, b0, b1):
    x, row, real = _scores(s, b0, b1)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    lse = (top + x.sub_(top).exp_().sum(-1, keepdim=True).log())[..., 0]            # [B][KV][queries][group]
    return lse.permute(0, 2, 1, 3).flatten(2)[real]


def _plain_weigh(s):
    """Weight of a cached token and head: the sum of its probabilities over the step's queries, and decay times what it had before
    (nothing for the step's own tokens)."""
    c = s["case"]
    page, KV = c["page"], c["kv_heads"]

    def part(s, b0, b1):
        x, row, _ = _scores(s, b0, b1)
        lse = s["lse"][row].unflatten(-1, (KV, -1)).permute(0, 2, 1, 3)[..., None]  # [B][KV][queries][group][1]
        lse = torch.where(lse == -math.inf, math.inf, lse)
        w = x.sub_(lse).exp_().sum((2, 3))                                          # [B][KV][L]
        lens = s["lens"][b0:b1].long()
        counts = (s["starts"][b0 + 1:b1 + 1] - s["starts"][b0:b1]).long()
        b, t = ((torch.arange(w.shape[-1], device=DEV) < lens[:, None]) & (counts > 0)[:, None]).nonzero(as_tuple=True)
        at = s["table"][b0 + b, t // page].long()
        before = s["weights"][at, :, t % page] if c["decay"] else torch.zeros(len(b), KV, device=DEV)
        before = torch.where((t < (lens - counts)[b])[:, None], c["decay"] * before, 0.0)
        s["out"][at, :, t % page] = before + w[b, :, t]
        return b[:0]

    _in_parts(s, part)
    return dict(weights=s["out"])


def _plain_evict(s):
    """A request past the limit keeps `budget` tokens of each head: the first `sinks`, the last `recent` and between them those of the
    largest weight (the earliest where several are), in their order, in pages from the ring's head; its old pages go behind the tail."""
    c = s["case"]
    page, KV, budget = c["page"], c["kv_heads"], c["budget"]
    table, held, free, ring = s["table"], s["held"].long(), s["free"], s["ring"]
    B, most = table.shape
    lens = s["lens"].long()
    each = -(-budget // page)
    over = lens > c["limit"]
    turn = over.cumsum(0) - over.long()
    served = over & ((turn + 1) * each <= ring[1] - ring[0])
    L = int(lens.max())
    t = torch.arange(L, device=DEV)
    at = table.long()[:, t // page]                                                 # [B][L]
    w = s["weights"][at, :, t % page].permute(0, 2, 1)                              # [B][KV][L]
    t3 = t[None, None]
    must = (t3 < c["sinks"]) | (t3 >= (lens - c["recent"])[:, None, None])
    w = torch.where(must, math.inf, w)
    w = torch.where(t3 < lens[:, None, None], w, -math.inf)
    # the budget-th largest weight; all above it, and the earliest of those equal to it
    place = min(budget, L)
    least = w.sort(-1, descending=True).values[..., place - 1:place]
    above, equal = w > least, w == least
    keep = above | (equal & (equal.cumsum(-1) <= place - above.sum(-1, keepdim=True)))
    kept = torch.full((B, KV, budget), -1, dtype=torch.int32, device=DEV)
    b, h, t = (keep & served[:, None, None]).nonzero(as_tuple=True)
    n = int(served.sum())
    kept[served] = t.int().reshape(n, KV, budget)
    which = served.nonzero()[:, 0]
    i = torch.arange(each, device=DEV)
    new = free[(ring[0] + turn[served][:, None] * each + i) % len(free)].long()     # [n][each]
    # bytes and weights of the kept tokens, from their old slots to the new ones
    i = torch.arange(budget, device=DEV)
    heads = torch.arange(KV, device=DEV)[:, None]
    old_t = kept[which].long()                                                      # [n][KV][budget]
    old_slot = table.long()[which[:, None, None], old_t // page] * page + old_t % page
    new_slot = (new[:, i // page] * page + i % page)[:, None].expand(-1, KV, -1)
    s["weights"][new_slot // page, heads, new_slot % page] = s["weights"][old_slot // page, heads, old_slot % page]
    flat, places = s["cache"].view(-1), _token_bytes(c["dim"])

    def bytes_of(slot):
        record = (slot // page * KV + heads) * (page // 16) + slot % page // 16
        return record[..., None] * (17 * c["dim"]) + places[slot % 16]

    flat[bytes_of(new_slot)] = flat[bytes_of(old_slot)]
    back = torch.where(served, held, 0)
    behind = back.cumsum(0) - back
    place = torch.arange(most, device=DEV)
    give = place < back[:, None]
    free[((ring[1] + behind[:, None] + place) % len(free))[give]] = table[give]
    out = table.clone()
    out[which] = -1
    out[which, :each] = new.int()
    k, v = (torch.where((s["slots"] >= 0)[:, None, None], _token_values(c, s["cache"], s["slots"].clamp(min=0), which), 0.0) for which in range(2))
    return dict(table=out, lens=torch.where(served, budget, lens).int(), held=torch.where(served, each, held).int(),
                ring=ring + torch.stack([served.sum() * each, back.sum()]), kept=kept, refused=(over & ~served).sum().int().reshape(1), free=free,
                weights=s["weights"], k=k, v=v)


# ------------------------------------------------------------------- work --
def work(c):
    if c["op"] == "norm":
        T, N = c["tokens"], c["hidden"]
        y, r = (4 if c[x] == "f32" else 2 for x in ("y", "residual"))
        gate = {"none": 0, "channel": 4 * N, "token": 4 * T * N}[c["gate"]]
        vectors = sum((c[x] != "none") * (2 if c["bias"] else 1) for x in ("post", "pre"))
        return dict(bytes=T * N * (y + 2 * r + 2) + gate + 4 * N * vectors, flops=T * N * 10)
    if c["op"] == "logprobs":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["rows"] * (c["vocab"] * size + 8 * c["count"] + 4 + 8 * c["top"]), flops=c["rows"] * c["vocab"] * 6)
    mean = (c["shortest"] + c["longest"]) / 2
    KV, D = c["kv_heads"], c["dim"]
    if c["op"] == "weigh":
        nq = min(c["queries"], mean)
        seen = mean if c["queries"] == 1 else mean - (nq - 1) / 2                    # cached tokens a query sees, on average
        read = mean
        if c["window"] and c["window"] < mean:
            reach = c["window"] + c["sinks"]
            read, seen = min(mean, reach + nq - 1), min(seen, reach)
        # keys that are seen, weights in (where they count) and out, queries and their sums
        return dict(bytes=c["batch"] * (read * KV * D * 17 / 32 + mean * KV * (8 if c["decay"] else 4) + nq * c["heads"] * (D * 2 + 4) + read / c["page"] * 4),
                    flops=2 * c["batch"] * nq * c["heads"] * seen * D)
    if c["shortest"] == c["longest"]:
        share, mean = 1.0, c["longest"]
    else:                                             # requests past the limit, and how long those are
        share, mean = (c["longest"] - c["limit"]) / (c["longest"] - c["shortest"] + 1), (c["limit"] + 1 + c["longest"]) / 2
    over = 1 + (c["batch"] - 1) * share
    # all weights of those requests; kept tokens and their weights in and out; the values read back
    return dict(bytes=over * KV * (mean * 4 + c["budget"] * (2 * D * 17 / 16 + 4 + 4) + c["budget"] * D * 17 / 16) + c["batch"] * c["budget"] * KV * 8 * D, flops=over * KV * mean * 4)


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    if case["op"] == "weigh" and 2 * case["batch"] * case["queries"] * case["heads"] * case["longest"] * case["dim"] > 6e12:
        return None
    return {"norm": _exact_norm, "logprobs": _exact_logprobs, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](case, prepare(case, seed))


def _exact_norm(c, s):
    def norm(x, kind, weight, bias):
        if kind == "rms":
            x = x / (x.square().sum(1, keepdim=True) / x.shape[1] + 1e-6).sqrt()
        elif kind == "layer":
            variance, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            x = (x - mean) / (variance + 1e-6).sqrt()
        x = x if weight is None else x * weight.double()
        return x if bias is None else x + bias.double()

    y = norm(s["y"].double(), c["post"], s["post_weight"], s["post_bias"])
    r = s["residual"].double() + c["scale"] * (y if s["gate"] is None else y * s["gate"].double())
    return dict(residual=r, x=norm(r, c["pre"], s["pre_weight"], s["pre_bias"]))


def _exact_logprobs(c, s):
    found = dict(logprobs=[], entropy=[], top_logprobs=[])
    step = max(1, (1 << 28) // c["vocab"])
    for at in range(0, c["rows"], step):
        x = s["logits"][at:at + step].double() * c["scale"]
        log_p = torch.log_softmax(x, 1)
        found["logprobs"].append(log_p.gather(1, s["tokens"][at:at + step].long()))
        found["entropy"].append(torch.special.entr(log_p.exp()).sum(1))
        if c["top"]:
            best = log_p.topk(min(c["top"], c["vocab"]), 1).values
            found["top_logprobs"].append(torch.nn.functional.pad(best, (0, c["top"] - best.shape[1]), value=-math.inf))
    return dict(top_tokens=None, **{k: torch.cat(v) if v else None for k, v in found.items()})


def _exact_values(records):
    """uint8 [pages][KV][page / 16][17 D] -> 64-bit K and V [KV][pages * page][D], each value by the place of its four bits."""
    D = records.shape[-1] // 17
    t = torch.arange(16, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)[None, :]
    each = 2 if D > 64 else 1
    group, i, c = d // 64, d % 64 // 8, d % 8
    start = (t // 8) * (D // 8) * 8 + (group // each) * 64 * each                   # in words
    k_word = start + ((t % 8 * 4 + i // 2) * each + group % each) * 2 + i % 2
    v_word = start + ((i * 4 + t % 8 // 2) * 2 + t % 2) * each + group % each
    found = []
    for word, base in ((k_word, 0), (v_word, 8 * D + D // 2)):
        byte = records[..., base + 4 * word + 2 * (c % 2) + c // 4]
        n = torch.where(c // 2 % 2 == 1, byte >> 4, byte & 15).double() - 8
        at = base + 8 * D + 2 * (t * (D // 64) + group)
        scale = records[..., torch.stack([at, at + 1], -1)].contiguous().view(torch.float16)[..., 0].double()
        found.append((n * scale).transpose(0, 1).flatten(1, 3))
    return found


def _exact_weigh(c, s):
    KV, D, page = c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        length, lo, hi = int(s["lens"][b]), int(s["starts"][b]), int(s["starts"][b + 1])
        pages = s["table"][b].long()[:(length + page - 1) // page]
        k = _exact_values(s["cache"][pages])[0][:, :length]
        t = torch.arange(length, device=DEV)
        at = length - (hi - lo) + torch.arange(hi - lo, device=DEV)[:, None]
        hide = t > at
        if c["window"]:
            hide |= (t <= at - c["window"]) & (t >= c["sinks"])
        q = s["q"][lo:hi].double().reshape(hi - lo, KV, -1, D)
        lse = s["lse"][lo:hi].double().reshape(hi - lo, KV, -1)
        for h in range(KV):
            x = torch.einsum("qgd,td->gqt", q[:, h], k[h]) * s["scale"] - lse[:, h].T[..., None]
            w = x.masked_fill(hide, -math.inf).exp().sum((0, 1))
            if c["decay"]:
                before = s["weights"][pages, h].flatten()[:length].double()
                w[:length - (hi - lo)] += c["decay"] * before[:length - (hi - lo)]
            whole = out[pages, h].flatten()
            whole[:length] = w
            out[pages, h] = whole.reshape(-1, page)
    return dict(weights=out)


def _exact_evict(c, s):
    page, KV, budget, sinks, recent = c["page"], c["kv_heads"], c["budget"], c["sinks"], c["recent"]
    each = -(-budget // page)
    room = int(s["ring"][1] - s["ring"][0])
    head = int(s["ring"][0])
    weights = s["weights"].double().clone()
    ks, vs, turn = [], [], 0
    for b in range(c["batch"]):
        length = int(s["lens"][b])
        if length <= c["limit"] or (turn + 1) * each > room:
            continue
        pages = s["table"][b].long()[:(length + page - 1) // page]
        k, v = _exact_values(s["cache"][pages])
        w = s["weights"][pages].transpose(0, 1).flatten(1)[:, :length].double()
        inner = torch.argsort(w[:, sinks:length - recent], dim=1, descending=True, stable=True)[:, :budget - sinks - recent] + sinks
        ends = torch.cat([torch.arange(sinks, device=DEV), torch.arange(length - recent, length, device=DEV)]).expand(KV, -1)
        keep = torch.cat([inner, ends], 1).sort(1).values
        ks.append(k.gather(1, keep[..., None].expand(-1, -1, k.shape[2])).transpose(0, 1))
        vs.append(v.gather(1, keep[..., None].expand(-1, -1, v.shape[2])).transpose(0, 1))
        t = torch.arange(budget, device=DEV)
        to = s["free"][(head + turn * each + torch.arange(each, device=DEV)) % len(s["free"])].long()[t // page]
        weights[to, :, t % page] = w.gather(1, keep).T
        turn += 1
    none = torch.zeros((c["batch"] - turn) * budget, KV, c["dim"], dtype=torch.float64, device=DEV)
    return dict(table=None, lens=None, held=None, ring=None, kept=None, refused=None, free=None, weights=weights,
                k=torch.cat([*ks, none]), v=torch.cat([*vs, none]))
