"""pn_logprobs where the roundings of a long row's sum all fall to one side.

Rows of equal logits but for a larger one at the front of each warp's part, so that all warps sum the same e = exp(-d)
over and over under a reference that stays.  With u = 2^-24: a thread adds 16 values at a time (two chains of 8) and one
such sum a turn, of which a row of V values and one block has V / 4096; then come the pair, 5 additions of lanes and 3 joins
of warps under equal references (two additions and a product by 1 each): a chain of V / 4096 + 8 + 1 + 5 + 9, below
V / 4096 + 32.  e errs by 2^-22 for ex2 and 4 u d for its argument (two roundings of d log2 e, and those of d where
it is a difference); the logarithm by 2 u of itself and the result, l, by u |l|.
"""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("vocab", [1 << 20, 1 << 19, 151936])
def test_equal_logits(vocab):
    from bit_weight_only_pn_gb300 import build, pn
    build.build()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 2 * sms + 1                                       # a block to a row
    d = torch.tensor([2.84753251, 2.66653885, 0.69626542, 2.68817939, 1.96617206, 1.52549183, 1.42319106, 2.02224075, 2.83572858,
                      2.13732911, 1.28842948, 1.39663221, 0.09426475, 1.53827943, 0.2073858, 0.21918973])
    d = torch.cat([d, torch.rand(rows - len(d), generator=torch.Generator().manual_seed(0)) * 3]).cuda()
    logits = torch.zeros(rows, vocab, device="cuda") - d[:, None]
    logits[:, 0:1024:128] = 0                                # the first value of each of eight warps
    got = pn.logprobs(logits, torch.full((rows,), 5, dtype=torch.int32, device="cuda"), top=1)
    d = d.double()
    S = 8 + (vocab - 8) * torch.exp(-d)
    want = -d - torch.log(S)
    off = (got.logprobs.double() - want).abs()
    limit = (vocab / 4096 + 32) * U + 2.0 ** -22 + 4 * U * d + 3 * U * want.abs()
    print(vocab, float((off / U).max()), float((off / limit).max()))
    assert bool((off <= limit).all()), (float((off / limit).max()), int((off > limit).sum()))
    entropy = torch.log(S) + (vocab - 8) * d * torch.exp(-d) / S
    off = (got.entropy.double() - entropy).abs()
    limit = 2 * limit * (d + 1) + 2 * U * entropy
    assert bool((off <= limit).all()), (float((off / limit).max()), int((off > limit).sum()))
    assert bool((got.top_tokens == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("rise", [1e-5, 0.02, 1.0, 60.0])
def test_rising_logits(dtype, rise):
    """A new largest logit in every turn of every warp: the contract's bound."""
    from bit_weight_only_pn_gb300 import build, pn
    build.build()
    vocab, rows = 1 << 19, 2 * torch.cuda.get_device_properties(0).multi_processor_count + 1
    logits = (torch.linspace(-rise, 0, vocab, dtype=torch.float64, device="cuda") * torch.linspace(0.5, 1, rows, device="cuda")[:, None]).to(dtype)
    tokens = torch.arange(rows, dtype=torch.int32, device="cuda") * (vocab // rows)
    got = pn.logprobs(logits, tokens, top=1)
    for r in range(0, rows, 19):
        x = logits[r].double()
        l = x - torch.logsumexp(x, 0)
        want = l[tokens[r]]
        limit = (vocab / 512 + 128) * U + 2.0 ** -22 * (2 * math.log(vocab) + 2 + x.max() - x[tokens[r]]) + 2 * U * want.abs()
        assert (got.logprobs[r].double() - want).abs() <= limit, (r, float((got.logprobs[r].double() - want).abs() / limit))
        entropy = -(l.exp() * l).sum()
        assert (got.entropy[r].double() - entropy).abs() <= 2 * (math.log(vocab) + 1) * ((vocab / 512 + 128) * U + 2.0 ** -22 * (math.log(vocab) + 2))
