"""Measured cases of the serving-step operators around the PN GEMV.

A speculative decoding step over PN weights runs, besides the GEMVs:

  plan       pages and slots for the step's tokens, from the request lengths (pn.kv_plan)
  append     per-head norms of queries and keys, position rotation, keys and values
             into a paged cache held in 4 bits (pn.kv_append; pn.kv_read reads it back)
  attention  the step's queries against that cache (pn.attention)
  verify     the drafted tokens against the target's probabilities (pn.verify)

``run`` computes an operator in plain torch operations (``own`` false) or through
the framework's entry points (``own`` true); ``exact`` restates it in 64 bits.

The cache.  uint8 [pages][kv_heads][page_size / 16][17 D]: a record holds 16
tokens of one head of D values: K codes (8 D bytes), K scales (D / 2), V codes
(8 D), V scales (D / 2).  Values are pn4t's: groups of 64 with a signed fp16
scale d and 4-bit codes n, value d (n - 8), eight codes to a 32-bit word (code c
in half c & 1, at bit 4 (c >> 1)).  With h = token / 8, groups two by two in
planes (one to a plane for D = 64), and word i of a group holding values
8 i .. 8 i + 7, the words lie in the order
  K  [h][plane][token % 8][i / 2][group in plane][i % 2]
  V  [h][plane][i][token % 8 / 2][token % 2][group in plane]
and the scales [token][group].
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step of a small server: latency of a single launch
        dict(name="plan_decode_8", op="plan", batch=8, most_new=1, longest=4096, page=16, capacity=8, finish=0.0),
        # a large batch of mixed prompts and decodes with finished requests: whole slot map rebuilt
        dict(name="plan_mixed_4096", op="plan", batch=4096, most_new=64, longest=8192, page=64, capacity=160000, finish=0.05),
        # one token of the 27B-class layer's attention: 6144 query and 1024 key columns as heads of 256
        dict(name="append_1", op="append", tokens=1, heads=24, kv_heads=4, dim=256, rotary=64, page=16, dtype="f32", norm=True, interleaved=False, fused=False, skip=0.0),
        # a verification batch out of one fused projection, half precision, no norms, odd token count
        dict(name="append_verify_37", op="append", tokens=37, heads=32, kv_heads=8, dim=64, rotary=64, page=32, dtype="f16", norm=False, interleaved=True, fused=True, skip=0.1),
        # a prompt chunk: the same layer as 48 heads of 128, bound by memory
        dict(name="append_prompt_8192", op="append", tokens=8192, heads=48, kv_heads=8, dim=128, rotary=128, page=64, dtype="f32", norm=True, interleaved=False, fused=False, skip=0.0),
        # the first tokens of one conversation: latency
        dict(name="attention_1_short", op="attention", batch=1, longest=130, shortest=130, queries=1, heads=24, kv_heads=4, dim=256, page=16, window=0, sinks=0),
        # one request with a very long cache: the split over its length
        dict(name="attention_1_long", op="attention", batch=1, longest=131072, shortest=131072, queries=1, heads=48, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # a decode batch of ragged lengths, the server's usual step
        dict(name="attention_64_ragged", op="attention", batch=64, longest=16384, shortest=1, queries=1, heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # one token and seven drafts for each request, a window and four first tokens that stay visible
        dict(name="attention_verify_window", op="attention", batch=24, longest=20000, shortest=500, queries=8, heads=48, kv_heads=8, dim=128, page=32, window=4096, sinks=4),
        # a prompt chunk against what is cached of it
        dict(name="attention_prompt_4096", op="attention", batch=1, longest=8192, shortest=8192, queries=4096, heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0),
        # one request, three drafts, a small vocabulary: latency
        dict(name="verify_1", op="verify", batch=1, drafts=3, vocab=32000, greedy_draft=True),
        # a batch with seven drafts each and the draft model's probabilities
        dict(name="verify_64", op="verify", batch=64, drafts=7, vocab=151936, greedy_draft=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attention", "attention", "attention", "verify"])
    if op == "plan":
        batch = _log(rng, 1, 4096)
        new = _log(rng, 1, 64)
        return dict(op=op, batch=batch, most_new=new, longest=_log(rng, 16, 8192), page=rng.choice([16, 32, 64, 128]),
                    capacity=batch * new + rng.randrange(64), finish=rng.choice([0.0, 0.05, 0.2]))
    if op == "append":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 6, 8])
        most = max(2, min(16384, 8192 * 48 * 128 // (heads * dim)))
        return dict(op=op, tokens=_log(rng, 1, most), heads=heads, kv_heads=kv, dim=dim, rotary=rng.choice([dim, dim, dim // 2, dim // 4]),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["f32", "f16"]), norm=rng.random() < 0.6,
                    interleaved=rng.random() < 0.3, fused=rng.random() < 0.5, skip=rng.choice([0.0, 0.1]))
    if op == "attention":
        dim = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 6, 8])
        kind = rng.choice(["one", "one", "drafts", "prompt"])
        queries = 1 if kind == "one" else rng.randint(2, 16) if kind == "drafts" else _log(rng, 17, 2048)
        batch = _log(rng, 1, 128) if kind != "prompt" else rng.randint(1, 4)
        # what the largest listed case reads, and a bound on the plain form's scores
        most = min(131072, 64 * 16384 * 8 * 128 // (batch * kv * dim), (1 << 30) // (batch * queries * kv * group))
        longest = max(queries, _log(rng, 1, max(2, most)))
        windowed = rng.random() < 0.3
        return dict(op=op, batch=batch, longest=longest, shortest=rng.choice([1, longest]), queries=queries, heads=kv * group, kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), window=_log(rng, 1, longest + 1) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0)
    vocab = _log(rng, 1000, 151936)
    batch = _log(rng, 1, 64)
    return dict(op=op, batch=batch, drafts=rng.randint(1, 7), vocab=vocab, greedy_draft=rng.random() < 0.4)


# ----------------------------------------------------------------- inputs --
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _generator(seed)
    return dict(case=case, **{"plan": _prepare_plan, "append": _prepare_append, "attention": _prepare_attention, "verify": _prepare_verify}[case["op"]](case, g))


def _randint(g, lo, hi, size):
    """Whole numbers from lo to hi, both included."""
    return torch.randint(lo, hi + 1, size, generator=g, device=DEV)


def _prepare_plan(c, g):
    batch, page = c["batch"], c["page"]
    lens = _randint(g, 0, c["longest"], (batch,))
    add = _randint(g, 1, c["most_new"], (batch,))
    add = torch.where(torch.rand(batch, generator=g, device=DEV) < c["finish"], -1, add)
    # pages in use; some requests hold one more, kept from drafts that were turned down
    held = (lens + page - 1) // page + (torch.rand(batch, generator=g, device=DEV) < 0.2)
    most_pages = (c["longest"] + c["most_new"]) // page + 2
    used = int(held.sum())
    pages = batch * (most_pages + 2)
    spare = int(0.36 * batch * c["most_new"] / page) + 1               # about what the step needs, so the last requests may be refused
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.zeros(batch, most_pages, dtype=torch.int32, device=DEV)
    place = torch.arange(most_pages, device=DEV).expand(batch, -1) < held[:, None]
    table[place] = order[:used].int()
    head = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
    free = torch.zeros(pages, dtype=torch.int32, device=DEV)
    free[(head + torch.arange(spare, device=DEV)) % pages] = order[used:used + spare].int()
    ring = torch.tensor([head, head + spare], dtype=torch.int64, device=DEV)
    return dict(lens=lens.int(), add=add.int(), held=held.int(), table=table, free=free, ring=ring)


def _prepare_append(c, g):
    T, H, KV, D, page = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    dtype = torch.float32 if c["dtype"] == "f32" else torch.float16
    rows = torch.randn(T, (H + 2 * KV) * D, generator=g, device=DEV)
    rows = rows * (0.5 + 2 * torch.rand(1, rows.shape[1], generator=g, device=DEV) ** 3)   # a few loud channels
    if c["fused"]:
        q, k, v = (x.unflatten(1, (-1, D)) for x in rows.to(dtype).split([H * D, KV * D, KV * D], dim=1))
    else:
        q, k, v = (x.to(dtype).contiguous().unflatten(1, (-1, D)) for x in rows.split([H * D, KV * D, KV * D], dim=1))
    start = int(torch.randint(0, 30000, (1,), generator=g, device=DEV))
    positions = start + torch.arange(T, device=DEV, dtype=torch.int32)
    # the tokens' pages lie in any order in a cache twice as large as they need
    pages = 2 * (T // page + 2)
    order = torch.randperm(pages, generator=g, device=DEV)
    at = start % page + torch.arange(T, device=DEV)
    slots = order[at // page] * page + at % page
    slots = torch.where(torch.rand(T, generator=g, device=DEV) < c["skip"], -1, slots)
    half = c["rotary"] // 2
    angle = torch.arange(start, start + T, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
    cos, sin = torch.zeros(start + T, half, device=DEV), torch.zeros(start + T, half, device=DEV)
    cos[start:], sin[start:] = angle.cos().float(), angle.sin().float()
    weights = [1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2)] if c["norm"] else [None, None]
    return dict(q=q, k=k, v=v, positions=positions, slots=slots, cos=cos, sin=sin, q_weight=weights[0], k_weight=weights[1],
                cache=torch.zeros(pages, KV, page // 16, 17 * D, dtype=torch.uint8, device=DEV))


def _prepare_attention(c, g):
    B, H, KV, D, page, nq = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], c["queries"]
    lens = _randint(g, c["shortest"], c["longest"], (B,))
    lens[0] = c["longest"]
    counts = lens.clamp(max=nq)                       # a request shorter than the others' drafts has fewer queries
    starts = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    starts[1:] = counts.cumsum(0)
    held = (lens + page - 1) // page
    most = int(held.max())
    used = int(held.sum())
    pages = used + 3
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.zeros(B, most, dtype=torch.int32, device=DEV)
    place = torch.arange(most, device=DEV).expand(B, -1) < held[:, None]
    table[place] = order[:used]
    cache = torch.empty(pages, KV, page // 16, 17 * D, dtype=torch.uint8, device=DEV)
    loud = 0.5 + 2 * torch.rand(2, KV, D, generator=g, device=DEV) ** 3
    step = max(1, (1 << 26) // (KV * page * D))       # pages at a time, for the memory that quantising takes
    for at in range(0, pages, step):
        n = min(step, pages - at)
        k, v = (loud[i, None, :, None] * torch.randn(n, KV, page, D, generator=g, device=DEV) for i in range(2))
        cache[at:at + n] = _records(*_quantise(k), *_quantise(v))
    q = torch.randn(int(starts[-1]), H, D, generator=g, device=DEV).half()
    return dict(q=q, cache=cache, table=table, lens=lens.int(), starts=starts, scale=1.5 / math.sqrt(D))


def _prepare_verify(c, g):
    B, K, V = c["batch"], c["drafts"], c["vocab"]
    logits = 2.0 * torch.randn(B, K + 1, V, generator=g, device=DEV)
    likely = _randint(g, 0, V - 1, (B, K + 1, 1))                # a token that the models lean to, more or less
    logits.scatter_add_(-1, likely, 9 + 9 * torch.rand(B, K + 1, 1, generator=g, device=DEV))
    target = torch.softmax(logits, -1)
    near = logits[:, :K] + 0.7 * torch.randn(B, K, V, generator=g, device=DEV)
    noise = -torch.log(-torch.log(torch.rand(B, K, V, generator=g, device=DEV).clamp(1e-7, 1 - 1e-7)))
    if c["greedy_draft"]:
        tokens, draft = near.argmax(-1), None
    else:
        tokens, draft = (near + noise).argmax(-1), torch.softmax(near, -1)
    counts = _randint(g, max(0, K - 2), K, (B,))
    uniforms = torch.rand(B, K + 1, generator=g, device=DEV)
    return dict(tokens=tokens.int(), target=target, draft=draft, uniforms=uniforms, counts=counts.int())


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


def _values(records):
    """uint8 [..., 17 D] records -> fp32 K and V [..., 16, D]."""
    D = records.shape[-1] // 17
    planes, each = _planes(D)
    lead = records.shape[:-1]
    c = torch.arange(8, device=records.device, dtype=torch.int32)
    shift = 16 * (c & 1) + 4 * (c >> 1)

    def values(codes, scales, shape, order):
        w = codes.contiguous().view(torch.int32)
        n = (w[..., None] >> shift) & 15
        m = len(lead)
        n = n.reshape(lead + shape + (8,)).permute(*range(m), *(m + i for i in order), m + len(order)).reshape(lead + (16, D // 64, 64))
        d = scales.contiguous().view(torch.float16).float().reshape(lead + (16, D // 64, 1))
        return (d * (n - 8).float()).reshape(lead + (16, D))

    k, kd, v, vd = records.split([8 * D, D // 2, 8 * D, D // 2], -1)
    return (values(k, kd, (2, planes, 8, 4, each, 2), (0, 2, 1, 4, 3, 5)),
            values(v, vd, (2, planes, 8, 4, 2, each), (0, 3, 4, 1, 5, 2)))


# -------------------------------------------------------------------- run --
def run(state):
    if own:
        return {"plan": _own_plan, "append": _own_append, "attention": _own_attention, "verify": _own_verify}[state["case"]["op"]](state)
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention, "verify": _plain_verify}[state["case"]["op"]](state)


def _own_plan(s):
    from bit_weight_only_pn_gb300 import pn
    p = pn.kv_plan(s["lens"], s["add"], s["held"], s["table"], s["free"], s["ring"], page_size=s["case"]["page"], capacity=s["case"]["capacity"])
    return dict(slots=p.slots, positions=p.positions, requests=p.requests, starts=p.starts, lens=p.lens, held=p.held, ring=p.ring, refused=p.refused,
                table=s["table"], free=s["free"])


def _own_append(s):
    from bit_weight_only_pn_gb300 import pn
    q = pn.kv_append(s["q"], s["k"], s["v"], s["cache"], s["slots"], s["positions"], s["cos"], s["sin"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                     eps=1e-6, interleaved=s["case"]["interleaved"])
    k, v = pn.kv_read(s["cache"], s["slots"])
    return dict(q=q, k=k, v=v)


def _own_attention(s):
    from bit_weight_only_pn_gb300 import pn
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = pn.AttentionWorkspace()
    out, lse = pn.attention(s["q"], s["cache"], s["table"], s["lens"], s["starts"], max_queries=c["queries"], scale=s["scale"], window=c["window"],
                            sinks=c["sinks"], workspace=s["workspace"], return_lse=True)
    return dict(out=out, lse=lse)


def _own_verify(s):
    from bit_weight_only_pn_gb300 import pn
    accepted, tokens = pn.verify(s["tokens"], s["target"], s["draft"], s["uniforms"], counts=s["counts"])
    return dict(accepted=accepted, tokens=tokens)


def _plain_plan(s):
    """Requests take pages from the ring in order, each all that it needs or none; finished ones (add < 0) give theirs back."""
    page, T = s["case"]["page"], s["case"]["capacity"]
    lens, add, held, table, free, ring = (s[k] for k in ("lens", "add", "held", "table", "free", "ring"))
    B, most = table.shape
    new = add.clamp(min=0)
    starts = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    starts[1:] = new.cumsum(0)
    done = add < 0
    want = (lens + new + page - 1) // page
    fits = ~done & (want <= most) & (starts[1:] <= T)
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    before = need.cumsum(0) - need
    served = fits & ((need == 0) | (before + need <= ring[1] - ring[0]))
    need = torch.where(served, need, 0)
    place = torch.arange(most, device=DEV)
    fresh = (place >= held[:, None]) & (place < (held + need)[:, None])
    taken = free[(ring[0] + before[:, None] + place - held[:, None]) % len(free)]
    table.copy_(torch.where(fresh, taken, table))
    back = torch.where(done, held, 0)
    behind = back.cumsum(0) - back
    give = place < back[:, None]
    # pages given back follow the ring's tail; the rest of the scatter lands in a spare place
    at = torch.where(give, (ring[1] + behind[:, None] + place) % len(free), len(free))
    free.copy_(torch.cat([free, free[:1]]).scatter(0, at.flatten(), table.flatten())[:-1])
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    b = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp(max=B - 1)
    real = t < starts[-1]
    positions = torch.where(real & served[b], lens[b] + t - starts[b], -1)
    slots = torch.where(positions >= 0, table[b, (positions // page).clamp(0, most - 1)].long() * page + positions % page, -1)
    return dict(slots=slots, positions=positions.int(), requests=torch.where(real, b, -1).int(), starts=starts,
                lens=torch.where(done, 0, lens + torch.where(served, new, 0)).int(), held=torch.where(done, 0, held + need).int(),
                ring=ring + torch.stack([need.sum(), back.sum()]), refused=(~done & ~served).sum().int().reshape(1), table=table, free=free)


def _turn(x, cos, sin, interleaved):
    """x [T][heads][D] with its first 2 * cos.shape[-1] values rotated."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = r[..., :half], r[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_norm(x, weight, eps):
    """x / sqrt(mean(x^2) + eps) * weight; the squares are added pairwise, the upper half to the lower, until one is left."""
    if weight is None:
        return x
    p = x * x
    while p.shape[-1] > 1:
        p = p[..., :p.shape[-1] // 2] + p[..., p.shape[-1] // 2:]
    return x * (1.0 / torch.sqrt(p * (1.0 / x.shape[-1]) + eps)) * weight


def _plain_append(s):
    cos, sin = s["cos"][s["positions"]], s["sin"][s["positions"]]
    q, k = (_turn(_plain_norm(s[x].float(), s[x + "_weight"], 1e-6), cos, sin, s["case"]["interleaved"]) for x in "qk")
    codes = [_quantise(x) for x in (k, s["v"].float())]
    kept = (s["slots"] >= 0)[:, None, None]
    k, v = (torch.where(kept, (d.float()[..., None] * (n.float() - 8).unflatten(-1, (-1, 64))).flatten(-2), 0.0) for n, d in codes)
    return dict(q=q.half(), k=k, v=v)


def _visible(c, lens, counts, most_q, length, where):
    """[B][most_q][length]: which cached tokens a request's queries see; its last query sits at the last token."""
    at = (lens - counts)[:, None, None] + torch.arange(most_q, device=where)[None, :, None]
    t = torch.arange(length, device=where)[None, None, :]
    see = (t <= at) & (t < lens[:, None, None])
    return see & ((t > at - c["window"]) | (t < c["sinks"])) if c["window"] else see


def _plain_attention(s):
    c = s["case"]
    B, H, KV, D, nq = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["queries"]
    lens, starts = s["lens"].long(), s["starts"].long()
    counts = starts[1:] - starts[:-1]
    k, v = _values(s["cache"][s["table"].long()])                                   # [B][pages][KV][page / 16][16][D]
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(B, KV, -1, D) for x in (k, v))
    L = k.shape[2]
    row = (starts[:-1, None] + torch.arange(nq, device=DEV)).clamp(max=len(s["q"]) - 1)
    q = s["q"].float()[row].reshape(B, nq, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(B, KV, -1, D)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).reshape(B, KV, nq, H // KV, L)
    x.masked_fill_(~_visible(c, lens, counts, nq, L, DEV)[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((torch.arange(L, device=DEV) < lens[:, None])[:, None, :, None], v, 0.0)
    out = (p.reshape(B, KV, -1, L) @ v).reshape(B, KV, nq, H // KV, D) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    real = torch.arange(nq, device=DEV) < counts[:, None]
    return dict(out=out.permute(0, 2, 1, 3, 4).reshape(B, nq, H, D)[real].half(), lse=lse.permute(0, 2, 1, 3).reshape(B, nq, H)[real])


def _plain_verify(s):
    """Accepts draft i while uniforms[i] * draft[i][x] < target[i][x]; then one token by the inverse of the cumulated
    weights max(target - draft, 0) (the target's alone after the last draft), held as whole multiples of 2^-42."""
    tokens, target, draft, uniforms, counts = (s[k] for k in ("tokens", "target", "draft", "uniforms", "counts"))
    B, K, V = target.shape[0], target.shape[1] - 1, target.shape[2]
    x = tokens.long()[..., None]
    p = target[:, :K].gather(-1, x)[..., 0]
    q = torch.ones_like(p) if draft is None else draft.gather(-1, x)[..., 0]
    i = torch.arange(K, device=DEV)
    ok = (uniforms[:, :K] * q < p) & (i < counts[:, None])
    accepted = ok.int().cumprod(-1).sum(-1)
    row = target[torch.arange(B, device=DEV), accepted]
    at = accepted.clamp(max=K - 1)
    turned = (accepted < counts)[:, None]
    j = torch.arange(V, device=DEV)
    if draft is None:
        rest = torch.where(turned & (j == tokens.long().gather(1, at[:, None])), 0.0, row)
    else:
        rest = torch.where(turned, row - draft[torch.arange(B, device=DEV), at], row)

    def whole(w):
        return torch.where(w > 0, w.clamp(max=1.0) * 2.0 ** 42, 0.0).round().to(torch.int64)

    rest = whole(rest)
    rest = torch.where(rest.sum(-1, keepdim=True) == 0, whole(row), rest)          # nothing left: the target itself
    sums = rest.cumsum(-1)
    total = sums[:, -1:]
    t = (uniforms[:, K:].double() * total.double()).floor().to(torch.int64).minimum(total - 1)
    pick = torch.where(total[:, 0] > 0, (sums <= t).sum(-1), -1).int()
    out = torch.where(i < accepted[:, None], tokens, -1)
    out = torch.cat([out, torch.full((B, 1), -1, dtype=torch.int32, device=DEV)], 1).scatter(1, accepted[:, None].long(), pick[:, None])
    return dict(accepted=accepted.int(), tokens=out)


# ------------------------------------------------------------------- work --
def work(c):
    if c["op"] == "plan":
        b = c["batch"]
        # lengths and held pages in and out, table entries and free pages that are taken (one for each request), the maps
        return dict(bytes=b * (4 + 4 + 4 + 4 + 4 + 4 + 8) + c["capacity"] * 16, flops=0)
    if c["op"] == "append":
        T, H, KV, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        size = 4 if c["dtype"] == "f32" else 2
        # q, k, v in; q out; the cache's bytes written, and the values read back
        return dict(bytes=T * ((H + 2 * KV) * D * size + H * D * 2 + KV * D * 17 / 16 * 2 + 2 * KV * D * 4 + 4 * c["rotary"] + 12), flops=T * (H + 2 * KV) * D * 8)
    if c["op"] == "attention":
        mean = (c["shortest"] + c["longest"]) / 2
        nq, D = min(c["queries"], mean), c["dim"]
        read = seen = mean if c["queries"] == 1 else mean - (nq - 1) / 2           # cached tokens a query sees, on average
        read = mean
        if c["window"] and c["window"] < mean:
            reach = c["window"] + c["sinks"]
            read, seen = min(mean, reach + nq - 1), min(seen, reach)
        return dict(bytes=c["batch"] * (read * c["kv_heads"] * D * 17 / 16 + nq * c["heads"] * (D * 4 + 4) + read / c["page"] * 4),
                    flops=4 * c["batch"] * nq * c["heads"] * seen * D)
    rows = 1 if c["greedy_draft"] else 2                                           # the whole rows that the last token is drawn from
    return dict(bytes=c["batch"] * (rows * c["vocab"] * 4 + c["drafts"] * 16), flops=c["batch"] * c["vocab"] * 3)


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    if case["op"] == "attention":
        return _exact_attention(case, prepare(case, seed))
    return None                                                                    # whole numbers alone


def _exact_append(c, s):
    out = {}
    slots = s["slots"]
    angle_c, angle_s = (s[x].double()[s["positions"].long()] for x in ("cos", "sin"))
    for name in "qkv":
        x = s[name].double()
        weight = s.get(name + "_weight")
        if name != "v":
            if weight is not None:
                x = x * (x.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * weight.double()
            R = c["rotary"]
            first = torch.arange(0, R, 2, device=DEV) if c["interleaved"] else torch.arange(R // 2, device=DEV)
            second = first + (1 if c["interleaved"] else R // 2)
            z = torch.complex(x[..., first], x[..., second]) * torch.complex(angle_c, angle_s)[:, None]
            x = x.clone()
            x[..., first], x[..., second] = z.real, z.imag
        if name != "q":
            y = x.reshape(*x.shape[:-1], -1, 64)
            # the largest value (the first of several), of whichever sign, at step -8
            d = (y.gather(-1, y.abs().argmax(-1, keepdim=True)) / -8).float().half().double()
            n = torch.round(y / torch.where(d == 0, 1.0, d)).clamp(-8, 7)
            x = torch.where((slots < 0)[:, None, None], 0.0, (n * d).reshape(x.shape))
        out[name] = x
    return out


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


def _exact_attention(c, s):
    flops = 4 * c["batch"] * c["queries"] * c["heads"] * c["longest"] * c["dim"]
    if flops > 6e12:
        return None
    KV, D, page = c["kv_heads"], c["dim"], c["page"]
    outs, lses = [], []
    for b in range(c["batch"]):
        length, lo, hi = int(s["lens"][b]), int(s["starts"][b]), int(s["starts"][b + 1])
        t = torch.arange(length, device=DEV)
        records = s["cache"][s["table"][b].long()[:(length + page - 1) // page]]    # [pages][KV][page / 16][17 D]
        k, v = (x[:, :length] for x in _exact_values(records))
        at = length - (hi - lo) + torch.arange(hi - lo, device=DEV)[:, None]
        hide = t > at
        if c["window"]:
            hide |= (t <= at - c["window"]) & (t >= c["sinks"])
        q = s["q"][lo:hi].double().reshape(hi - lo, KV, -1, D)
        out = torch.empty(hi - lo, c["heads"], D, dtype=torch.float64, device=DEV)
        lse = torch.empty(hi - lo, c["heads"], dtype=torch.float64, device=DEV)
        for h in range(KV):
            x = torch.einsum("qgd,td->gqt", q[:, h], k[h]) * s["scale"]
            x = x.masked_fill(hide, -math.inf)
            group = slice(h * x.shape[0], (h + 1) * x.shape[0])
            lse[:, group] = torch.logsumexp(x, -1).T
            out[:, group] = torch.einsum("gqt,td->qgd", torch.softmax(x, -1), v[h])
        outs.append(out)
        lses.append(lse)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
