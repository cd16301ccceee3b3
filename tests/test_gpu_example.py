"""The speculative decoding example: drafts leave the text alone and save steps."""
from __future__ import annotations

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_drafts_give_the_same_text():
    from bit_weight_only_pn_gb300 import build
    build.build()
    import speculative_step as s
    model = s.Model()
    prompts = [[7, 8, 9, 7, 8], list(range(100, 163)), [3]]
    plain, plain_steps = s.generate(model, prompts, 40, 0)
    again, _ = s.generate(model, prompts, 40, 0)
    assert plain == again and all(len(t) == 40 for t in plain)
    drafted, steps = s.generate(model, prompts, 40, 3)
    assert plain_steps == 39 and 10 <= steps <= 39
    # sums of one token's and of four tokens' products differ in order, so a near tie may part two texts, hardly all three
    assert sum(a == b for a, b in zip(plain, drafted)) >= 1
    sampled, _ = s.generate(model, prompts, 20, 3, greedy=False)
    assert all(0 <= x < s.VOCAB for t in sampled for x in t)
