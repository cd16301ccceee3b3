"""Decoding with a cache that keeps what is looked at, every step on the library's calls:

    kv_plan -> norm -> gemv_layer (q, k, v) -> kv_append -> attention -> kv_weigh -> gemv (output projection)
    -> norm -> gemv (vocabulary) -> logprobs -> kv_evict

for a batch of requests with a one-layer model.  A request that has more than `limit`
tokens in the cache is cut back to `budget` of them: the first, the last and those that
queries gave the most weight, each key/value head its own.

    python examples/bounded_cache.py [--limit 192] [--budget 128] [--new 300] [--batch 4]

prints the pages in use, the text's mean log probability with and without the limit, and
how many tokens of the two texts agree.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bit_weight_only_pn_gb300 import pn  # noqa: E402
from speculative_step import DIM, EPS, HEADS, HIDDEN, KV_HEADS, PAGE, POSITIONS, VOCAB, Model  # noqa: E402

SCALE = DIM ** -0.5
SINKS, RECENT = 4, 32


class State:
    """What a server keeps between steps."""

    def __init__(self, batch: int, longest: int):
        per_request = -(-longest // PAGE) + 1
        self.pages = batch * (per_request + -(-longest // PAGE))       # room for what is kept beside what it is kept of
        self.cache = pn.kv_cache(self.pages, PAGE, KV_HEADS, DIM)
        self.weights = pn.kv_weights(self.cache)
        self.table = torch.zeros(batch, per_request, dtype=torch.int32, device="cuda")
        self.free = torch.arange(self.pages, dtype=torch.int32, device="cuda")
        self.ring = torch.tensor([0, self.pages], device="cuda")
        self.lens, self.held, self.gone = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(3))


def step(model: Model, s: State, tokens: torch.Tensor, add: torch.Tensor, longest: int):
    """The step's tokens (request after request) join the cache; logits of all of them."""
    plan = pn.kv_plan(s.lens, add, s.held, s.table, s.free, s.ring, PAGE, len(tokens))
    # positions go on from the tokens that there have been, kept or not
    positions = plan.positions + s.gone[plan.requests.clamp(min=0).long()]
    stream = model.embedding[tokens]
    _, x = pn.norm(None, stream, eps=EPS)
    q, k, v = model.project((model.q, model.k, model.v), x)
    q = pn.kv_append(q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)), s.cache, plan.slots, positions,
                     model.cos, model.sin, model.q_norm, model.k_norm, EPS)
    a, lse = pn.attention(q, s.cache, s.table, plan.lens, plan.starts, longest, SCALE, workspace=model.attn_ws, return_lse=True)
    pn.kv_weigh(q, s.cache, s.table, plan.lens, plan.starts, longest, lse, SCALE, weights=s.weights, workspace=model.attn_ws)
    _, x = pn.norm(model.project((model.o,), a.flatten(1))[0], stream, eps=EPS)
    s.lens, s.held, s.ring = plan.lens, plan.held, plan.ring
    return model.project((model.head,), x)[0], plan.starts


def generate(model: Model, prompts: list[list[int]], new: int, limit: int, budget: int):
    """`new` greedy tokens for each prompt (at most 16).  Returns (texts, their log probabilities [batch][new], most pages held by a request)."""
    batch, longest = len(prompts), max(map(len, prompts))
    if longest + new > POSITIONS:
        raise ValueError("longer than the table of positions")
    s = State(batch, min(max(limit + 1, longest + 1), longest + new) + PAGE)
    counts = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    tokens, add = torch.tensor([t for p in prompts for t in p], device="cuda"), counts
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    texts, logprobs, most = [], [], torch.zeros((), dtype=torch.int32, device="cuda")
    for _ in range(new):
        logits, starts = step(model, s, tokens, add, int(longest) if not texts else 1)
        last = logits[starts[1:].long() - 1]
        p = pn.logprobs(last, top=1)
        texts.append(p.top_tokens[:, 0])
        logprobs.append(p.top_logprobs[:, 0])
        e = pn.kv_evict(s.cache, s.weights, s.table, s.lens, s.held, s.free, s.ring, limit, budget, SINKS, RECENT)
        s.gone = s.gone + s.lens - e.lens
        s.table, s.lens, s.held, s.ring = e.table, e.lens, e.held, e.ring
        most = torch.maximum(most, s.held.max())
        tokens, add = p.top_tokens[:, 0].long(), one
    held = int(s.held.sum())
    if int(s.ring[1] - s.ring[0]) + held != s.pages or model.attn_ws.status() or model.gemv_ws.status():
        raise RuntimeError("a page was lost or a device-side wait gave up")
    return torch.stack(texts, 1).tolist(), torch.stack(logprobs, 1), int(most)


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--limit", type=int, default=192)
    p.add_argument("--budget", type=int, default=128)
    p.add_argument("--new", type=int, default=300)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args()
    if not 1 <= a.batch <= 16 or not SINKS + RECENT <= a.budget <= a.limit:
        p.error(f"batch must be 1 .. 16 and {SINKS + RECENT} <= budget <= limit")
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(VOCAB, (20 + 37 * b,), generator=g).tolist() for b in range(a.batch)]
    texts = {}
    for limit, budget in ((POSITIONS, POSITIONS), (a.limit, a.budget)):
        generate(model, prompts, 3, limit, budget)                  # first use of each shape
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        texts[limit], logprobs, most = generate(model, prompts, a.new, limit, budget)
        torch.cuda.synchronize()
        print(f"limit {limit}: {a.batch} x {a.new} tokens in {(time.perf_counter() - t0) * 1e3:.1f} ms, at most {most} pages to a request, "
              f"mean log probability {logprobs.mean():.4f}")
    whole, cut = texts.values()
    same = sum(x == y for u, v in zip(whole, cut) for x, y in zip(u, v))
    print(f"tokens that agree: {same} of {a.batch * a.new}")


if __name__ == "__main__":
    main()
