"""pn_kv_evict for several layers that share page tables and a ring: a call for each on the first one's inputs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_step_operators import cuda, evict_case, ref_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pn():
    from bit_weight_only_pn_gb300 import build, pn as module
    build.build()
    return module


def check_layer(pn, case, got, before, after, limit, budget, sinks, recent):
    cache, weights, table, lens, held, free, ring = case
    page = cache.shape[2] * 16
    ring_after = free.copy()
    want = ref_evict(weights, table, lens, held, ring_after, ring, page, limit, budget, sinks, recent)
    for name in got._fields:
        assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), name
    new_cache, new_weights = after
    for b in np.flatnonzero(want["kept"][:, 0, 0] >= 0):
        t = np.arange(budget)
        new = want["table"][b, t // page].astype(np.int64) * page + t % page
        k_new, v_new = pn.kv_read(new_cache, cuda(new))
        for h in range(cache.shape[1]):
            p = want["kept"][b, h]
            old = table[b, p // page].astype(np.int64) * page + p % page
            k_old, v_old = pn.kv_read(before, cuda(old))
            assert torch.equal(k_new[:, h], k_old[:, h]) and torch.equal(v_new[:, h], v_old[:, h])
            assert np.array_equal(new_weights.cpu().numpy()[new // page, h, new % page], weights[old // page, h, old % page])
    return want, ring_after


@pytest.mark.parametrize("lens,kv,D,page,limit,budget,sinks,recent,spare", [
    ([200, 500, 90], 2, 128, 32, 80, 47, 4, 8, None), ([90, 80, 70, 100], 2, 64, 16, 64, 40, 2, 2, 7), ([700, 20, 650], 1, 256, 64, 100, 100, 0, 30, None)])
@pytest.mark.parametrize("captured", [False, True])
def test_three_layers(pn, lens, kv, D, page, limit, budget, sinks, recent, spare, captured):
    first = evict_case(lens, kv, D, page, budget, spare)
    rng = np.random.default_rng(7)
    layers = [first]
    for _ in range(2):
        cache = first[0].copy()
        cache[..., :8 * D] = rng.integers(0, 256, cache[..., :8 * D].shape)
        layers.append((cache, rng.random(first[1].shape).astype(np.float32), *first[2:]))
    table, lens_, held, ring = (cuda(first[i]) for i in (2, 3, 4, 6))
    free = cuda(first[5])
    caches, weights = [cuda(c[0]) for c in layers], [cuda(c[1]) for c in layers]
    before = [c.clone() for c in caches]

    def step():
        return [pn.kv_evict(c, w, table, lens_, held, free, ring, limit, budget, sinks, recent) for c, w in zip(caches, weights)]

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graph.replay()
    else:
        got = step()
    for i, case in enumerate(layers):
        want, ring_after = check_layer(pn, case, got[i], before[i], (caches[i], weights[i]), limit, budget, sinks, recent)
        assert np.array_equal(free.cpu().numpy(), ring_after)
        for name in ("table", "lens", "held", "ring", "refused"):
            assert torch.equal(getattr(got[i], name), getattr(got[0], name))
    # the next step begins from that state: nothing is past the limit, and nothing changes
    state = got[0]
    if int(state.refused) == 0:
        held_cache = [c.clone() for c in caches]
        held_free, held_weights = free.clone(), [w.clone() for w in weights]
        for c, w in zip(caches, weights):
            again = pn.kv_evict(c, w, state.table, state.lens, state.held, free, state.ring, limit, budget, sinks, recent)
            for name in ("table", "lens", "held", "ring"):
                assert torch.equal(getattr(again, name), getattr(state, name))
            assert int(again.refused) == 0 and bool((again.kept == -1).all())
        assert all(torch.equal(a, b) for a, b in zip(caches + weights + [free], held_cache + held_weights + [held_free]))


def test_narrow_requests_in_wide_tables(pn):
    """Tables wider than any request needs, lengths below 0 and past the table: what is kept is the same."""
    case = list(evict_case([1281, 60, 300], 2, 64, 16, 50, seed=3))
    narrow = [cuda(c) for c in case]
    got = pn.kv_evict(*narrow, 200, 50, 4, 9)
    wide = [cuda(c) for c in case]
    wide[2] = torch.full((3, 8192), -1, dtype=torch.int32, device="cuda")
    wide[2][:, :case[2].shape[1]] = cuda(case[2])
    more = pn.kv_evict(*wide, 200, 50, 4, 9)
    assert torch.equal(more.kept, got.kept) and torch.equal(more.lens, got.lens) and torch.equal(more.ring, got.ring)
    assert torch.equal(more.table[:, :4], got.table[:, :4]) and torch.equal(wide[1], narrow[1]) and torch.equal(wide[0], narrow[0])
    case[3] = np.array([-5, 1 << 30, 300], np.int32)         # as many as the table has room for
    odd = [cuda(c) for c in case]
    got = pn.kv_evict(*odd, 200, 50, 4, 9)
    room = case[2].shape[1] * 16
    assert got.lens.tolist() == [-5, 50, 50] and bool((got.kept[0] == -1).all())
    assert got.kept[1, :, -9:].tolist() == [list(range(room - 9, room))] * 2
