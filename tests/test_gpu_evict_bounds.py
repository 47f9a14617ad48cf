"""The bound of an eviction: a length above it ends there, and is cut to the budget
all the same; any bound at or above the lengths gives the same result."""

import numpy as np
import pytest

import gguf_block_quant_dequant_amd as g
from tests.serving_util import TYPES, dev, host
from tests.test_gpu_kv_cache import check_evict, evict_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(TYPES))
def test_bounds_at_and_above_the_lengths(kind):
    # each way of holding the keys for the same lengths
    for max_len in (200, 201, 4096, 5000, 9000, 20000, 40000, 1 << 30):
        d = evict_case(np.random.default_rng(90), kind, [200, 120, 0, 64, 65], 32)
        check_evict(d, 64, 8, max_len=max_len)


def test_sequences_past_the_bound_lose_their_last_tokens():
    # 100 of 200 tokens looked at, the newest eight of those protected: none of
    # the last hundred is left, whatever its weight or age
    d = evict_case(np.random.default_rng(91), "bf16", [200], 32, hkv=2)
    at = np.arange(200)
    page, slot = d["table"][0][at // 32], at % 32
    d["pos"][page, :, slot] = at[:, None]
    d["cache"].pos.copy_(dev(d["pos"]))
    check_evict(d, 64, 8, max_len=100)
    left = host(d["cache"].pos)[page[:64], :, slot[:64]]
    for h in range(2):
        assert set(range(92, 100)) <= set(left[:, h].tolist()) and left[:, h].max() == 99


def test_lengths_past_the_table_row():
    d = evict_case(np.random.default_rng(92), "f16", [128, 128], 32)
    for budget, moved in ((50, True), (128, False), (300, False)):
        n = dev(np.array([1000, 128], np.int32))
        before = host(d["cache"].k)
        g.gguf_kv_evict(d["cache"], dev(d["table"]), n, 2000, budget, recent=4)
        assert host(n).tolist() == [budget, min(budget, 128)]
        assert np.array_equal(host(d["cache"].k), before) != moved
