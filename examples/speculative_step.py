"""Speculative decoding with a one-layer model, every step on the library's calls:

    kv_plan -> gemv_layer (q, k, v) -> kv_append -> attention -> gemv (output projection, vocabulary) -> verify

for a batch of requests of unequal lengths whose keys and values live in pages of
the 4-bit cache.  Drafts come from the request's own text: what followed the last
token where it stood before.  Prompts go through the same calls, their projections
through ``prefill``.

    python examples/speculative_step.py [--drafts 3] [--new 200] [--batch 4]

generates with and without drafts from random weights (a layer small beside the
embedding, so that texts come round) and prints the tokens per step.  With greedy
targets both give the same text, but for near ties of the largest logit: the
products of one token and of several are added in different orders.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_only_pn_gb300 import pn  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE, VOCAB, POSITIONS = 640, 8, 2, 64, 16, 400, 4096
EPS = 1e-6


class Model:
    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rows(pn_type, n, k, size=1.0):
            return pn_type, pn.pack(pn_type, torch.randn(n, k, device="cuda", generator=g) * (size / k ** 0.5)), k

        self.embedding = torch.randn(VOCAB, HIDDEN, device="cuda", generator=g)
        self.q, self.k, self.v = rows(pn.PN3T, HEADS * DIM, HIDDEN), rows(pn.PN4T, KV_HEADS * DIM, HIDDEN), rows(pn.PN4T, KV_HEADS * DIM, HIDDEN)
        self.o, self.head = rows(pn.PN4T, HIDDEN, HEADS * DIM, 0.3), rows(pn.PN3T, VOCAB, HIDDEN)
        self.q_norm, self.k_norm = torch.ones(DIM, device="cuda"), torch.ones(DIM, device="cuda")
        angle = torch.arange(POSITIONS, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, DIM, 2, device="cuda") / DIM)
        self.cos, self.sin = angle.cos(), angle.sin()
        self.gemv_ws, self.attn_ws = pn.Workspace(VOCAB), pn.AttentionWorkspace()

    def project(self, weights, x: torch.Tensor):
        """x [tokens][K] times each of `weights`: one launch for a step's few tokens, the prefill GEMM for a prompt's."""
        x = x.half().contiguous()
        if len(x) > 16:
            return [pn.prefill(t, W, k, x, workspace=self.gemv_ws) for t, W, k in weights]
        ys = [torch.empty(len(x), len(W), device="cuda") for _, W, _ in weights]
        return pn.gemv_layer([(t, W, k, x, y) for (t, W, k), y in zip(weights, ys)], len(x), workspace=self.gemv_ws)

    def logits(self, tokens: torch.Tensor, plan: pn.KvPlan, cache: torch.Tensor, table: torch.Tensor, longest: int) -> torch.Tensor:
        """Logits of a step's tokens (request after request, as planned); keys and values join the cache."""
        x = self.embedding[tokens]
        norm = lambda a: a * torch.rsqrt(a.square().mean(-1, keepdim=True) + EPS)
        q, k, v = self.project((self.q, self.k, self.v), norm(x))
        q = pn.kv_append(q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)), cache, plan.slots,
                         plan.positions, self.cos, self.sin, self.q_norm, self.k_norm, EPS)
        a = pn.attention(q, cache, table, plan.lens, plan.starts, longest, DIM ** -0.5, workspace=self.attn_ws)
        x = x + self.project((self.o,), a.flatten(1))[0]
        return self.project((self.head,), norm(x))[0]


def drafts_from_text(text: torch.Tensor, length: torch.Tensor, count: int) -> torch.Tensor:
    """[batch][count] tokens that followed the latest earlier place of each request's last token (0 where there is none)."""
    at = torch.arange(text.shape[1], device="cuda")
    last = text.gather(1, length[:, None] - 1)
    seen = torch.where((text == last) & (at < length[:, None] - 1), at, -1).amax(1)
    place = seen[:, None] + 1 + torch.arange(count, device="cuda")
    ok = (seen[:, None] >= 0) & (place < length[:, None])
    return torch.where(ok, text.gather(1, place.clamp(max=text.shape[1] - 1)), 0).int()


def generate(model: Model, prompts: list[list[int]], new: int, drafts: int, greedy: bool = True, seed: int = 0):
    """`new` tokens for each prompt (at most 16 tokens a step: len(prompts) * (drafts + 1)).  Returns (text of each request, steps)."""
    batch, width = len(prompts), max(map(len, prompts)) + new + drafts + 1
    per_request = -(-width // PAGE) + 1
    pages = batch * per_request
    cache = pn.kv_cache(pages, PAGE, KV_HEADS, DIM)
    table = torch.zeros(batch, per_request, dtype=torch.int32, device="cuda")
    free, ring = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.tensor([0, pages], device="cuda")
    lens, held = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(seed)

    def probabilities(logits):
        if greedy:
            return torch.nn.functional.one_hot(logits.argmax(-1), VOCAB).float()
        return logits.softmax(-1)

    # the prompts: all tokens in one step, the last one's logits give the first new token
    counts = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    total = sum(map(len, prompts))
    plan = pn.kv_plan(lens, counts, held, table, free, ring, PAGE, total)
    logits = model.logits(torch.tensor([t for p in prompts for t in p], device="cuda"), plan, cache, table, max(map(len, prompts)))
    none = torch.zeros(batch, 0, dtype=torch.int32, device="cuda")
    last = logits[plan.starts[1:].long() - 1]
    _, out = pn.verify(none, probabilities(last)[:, None], None, torch.rand(batch, 1, device="cuda", generator=g))
    text = torch.zeros(batch, width + drafts + 1, dtype=torch.int64, device="cuda")
    for b, p in enumerate(prompts):
        text[b, :len(p)] = torch.tensor(p, device="cuda")
    length = counts.long() + 1
    text.scatter_(1, length[:, None] - 1, out.long())
    start, steps = counts.long(), 0
    add = torch.full((batch,), drafts + 1, dtype=torch.int32, device="cuda")
    while True:
        done = length - start >= new
        if bool(done.all()):
            break
        # a request that is done adds no more tokens, but keeps its rows, so that every step has the same shape
        tokens = drafts_from_text(text, length, drafts)
        plan = pn.kv_plan(plan.lens, torch.where(done, 0, add), plan.held, table, free, plan.ring, PAGE, batch * (drafts + 1))
        rows = torch.cat([text.gather(1, length[:, None] - 1), tokens.long()], 1)
        place = (plan.starts[:-1].long()[:, None] + torch.arange(drafts + 1, device="cuda")).clamp(max=batch * (drafts + 1) - 1)
        step_tokens = torch.zeros(batch * (drafts + 1), dtype=torch.int64, device="cuda")
        step_tokens.scatter_(0, place[~done].flatten(), rows[~done].flatten())
        logits = model.logits(step_tokens, plan, cache, table, drafts + 1)
        accepted, out = pn.verify(tokens, probabilities(logits[place]), None, torch.rand(batch, drafts + 1, device="cuda", generator=g))
        took = torch.where(done, 0, accepted.long() + 1)
        at = length[:, None] + torch.arange(drafts + 1, device="cuda")
        text.scatter_(1, at, torch.where((out >= 0) & ~done[:, None], out.long(), text.gather(1, at)))
        length = length + took
        # the cache keeps the last token's and the accepted drafts' entries; those behind them are written over
        plan = plan._replace(lens=torch.where(done, plan.lens, plan.lens - drafts + accepted))
        steps += 1
    plan = pn.kv_plan(plan.lens, torch.full_like(add, -1), plan.held, table, free, plan.ring, PAGE, 0)
    if int(plan.ring[1] - plan.ring[0]) != pages or model.attn_ws.status() or model.gemv_ws.status():
        raise RuntimeError("a page was lost or a device-side wait gave up")
    text, start = text.tolist(), start.tolist()
    return [t[s:s + new] for t, s in zip(text, start)], steps


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--drafts", type=int, default=3)
    p.add_argument("--new", type=int, default=200)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args()
    if a.batch * (a.drafts + 1) > 16:
        p.error("batch * (drafts + 1) must be at most 16")
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(VOCAB, (5 + 37 * b,), generator=g).tolist() for b in range(a.batch)]
    texts = {}
    for drafts in dict.fromkeys((0, a.drafts)):
        generate(model, prompts, 4, drafts)                     # first use of each shape
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        texts[drafts], steps = generate(model, prompts, a.new, drafts)
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t0) * 1e3
        print(f"{drafts} drafts: {a.batch} x {a.new} tokens in {steps} steps, {(a.new - 1) / max(steps, 1):.2f} tokens a step, {ms:.1f} ms")
    if a.drafts:
        same = sum(x == y for x, y in zip(texts[0], texts[a.drafts]))
        print(f"same text with and without drafts: {same} of {a.batch} requests")


if __name__ == "__main__":
    main()
