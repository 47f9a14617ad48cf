"""Positions of tokens appended after an eviction: given, they are the newest; left
out, they are the slots, which an eviction starts again at the budget."""

import numpy as np
import pytest

import gguf_block_quant_dequant_amd as g
from oracle.serving import evict_moves
from tests.serving_util import TYPES, dev, host, make

BUDGET, RECENT, LENGTH = 64, 8, 200


def test_slots_as_positions_lose_the_newest_token():
    rng = np.random.default_rng(1)
    weight, pos = rng.uniform(1, 2, LENGTH), np.arange(LENGTH)
    kept, _, _ = evict_moves(weight, pos, BUDGET, RECENT)
    weight, pos = np.append(weight[kept], 0.0), pos[kept]
    for new, stays in ((LENGTH, True), (BUDGET, False)):   # its position, its slot
        kept, _, _ = evict_moves(weight, np.append(pos, new), BUDGET, RECENT)
        assert (BUDGET in kept) == stays


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("given", [True, False])
def test_append_between_evictions(kind, given):
    rng = np.random.default_rng(2)
    d = make(rng, TYPES[kind], [LENGTH], 7, 2, 2, 64, 32, poisoned=False, planes=True)
    cache, t, n = d["cache"], dev(d["table"]), dev(d["lengths"])
    at = np.arange(LENGTH)
    d["pos"][d["table"][0][at // 32], :, at % 32] = at[:, None]
    cache.weight.copy_(dev(d["weight"] + np.float32(1.0)))
    cache.pos.copy_(dev(d["pos"]))
    g.gguf_kv_evict(cache, t, n, LENGTH, BUDGET, recent=RECENT)
    k = dev(rng.standard_normal((1, 128)).astype(np.float32))
    g.gguf_kv_append(cache, k, k, t, n, pos=dev(np.array([LENGTH], np.int32)) if given else None)
    n += 1
    new = LENGTH if given else BUDGET
    assert host(cache.pos)[d["table"][0][BUDGET // 32], :, BUDGET % 32].tolist() == [new, new]
    before, pos = host(cache.weight), host(cache.pos)
    g.gguf_kv_evict(cache, t, n, BUDGET + 1, BUDGET, recent=RECENT)
    assert host(n).tolist() == [BUDGET]
    at = np.arange(BUDGET + 1)
    page, slot = d["table"][0][at // 32], at % 32
    for h in range(2):
        p = pos[page, h, slot]
        kept, _, _ = evict_moves(before[page, h, slot], p, BUDGET, RECENT)
        left = host(cache.pos)[page[:BUDGET], h, slot[:BUDGET]]
        assert sorted(left.tolist()) == sorted(p[kept].tolist())
        assert (LENGTH in left.tolist()) == given
