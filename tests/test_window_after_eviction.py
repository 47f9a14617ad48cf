"""A window over a cache that evictions have cut: windows count slots, whose order
an eviction gives up; a window of positions is what an eviction with budget and
recent equal to it leaves. The oracle on the CPU, the library against it."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.serving import attend_f64, evict_moves, kv_values_f64, sequence_f64
from tests.serving_util import DEV, TYPES, U, attend_reference, check_bound, dev, host, make


def evicted_positions(steps, budget, recent, rng):
    """(token, positions in slot order) of a sequence cut to budget after every token."""
    pos, weight = np.zeros(0, int), np.zeros(0)
    for t in range(steps):
        pos, weight = np.append(pos, t), np.append(weight, 0.0)
        weight = weight + rng.random(len(weight))
        _, src, dst = evict_moves(weight, pos, budget, recent)
        pos[dst], weight[dst] = pos[src], weight[src]
        pos, weight = pos[:budget], weight[:budget]
        yield t, pos


def test_the_last_slots_are_not_the_newest_tokens():
    for t, pos in evicted_positions(200, 64, 8, np.random.default_rng(1)):
        assert set(range(max(0, t - 7), t + 1)) <= set(pos.tolist())   # the protected ones are somewhere
        same = set(pos[-16:].tolist()) == {x for x in pos.tolist() if x > t - 16}
        assert same == (t < 64), t   # until the first eviction


@pytest.mark.parametrize("window", [1, 7, 64])
def test_budget_and_recent_of_the_window_keep_its_positions(window):
    for t, pos in evicted_positions(200, window, window, np.random.default_rng(2)):
        assert sorted(pos.tolist()) == list(range(max(0, t - window + 1), t + 1))


def by_position(k, v, pos, q, window, scale):
    """Attention over the positions > max - window of one head's slots: (out, bound
    as in attend_reference)."""
    seen = np.flatnonzero(pos > pos.max() - window)
    out, p = attend_f64(q, k[seen], v[seen], scale)
    mag = scale * (np.abs(k[seen]) @ np.abs(q.astype(np.float64))).max()
    ew = (4 * U + 2.0 ** -22 + 3 * len(q) * U) * mag + 4 * U * mag + 4 * U + 2.0 ** -22
    return out, (2 * ew + (8 * len(p) + 128) * U) * (p @ np.abs(v[seen])) + 1e-30


def planes(d, rng):
    """Distinct positions in a mixed order, as evictions leave them, and weights."""
    d["weight"] = rng.uniform(0, 2, d["weight"].shape).astype(np.float32)
    for s, n in enumerate(d["lengths"]):
        at = np.arange(n)
        for h in range(d["hkv"]):
            d["pos"][d["table"][s][at // d["ps"]], h, at % d["ps"]] = rng.permutation(n)
    d["cache"].weight.copy_(dev(d["weight"]))
    d["cache"].pos.copy_(dev(d["pos"]))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 30, 100])
@pytest.mark.parametrize("kind", list(TYPES))
def test_position_window_by_eviction(kind, window):
    rng = np.random.default_rng([window, 60])
    lengths = [200, 90, 130, 0]
    d = make(rng, TYPES[kind], lengths, 7, 4, 2, 64, 32, poisoned=False, planes=True)
    planes(d, rng)
    args = (d["type"], d["n_pages"], 2, 64, 32)
    K, V = kv_values_f64(d["k"], *args, False), kv_values_f64(d["v"], *args, True)
    want, bound = np.zeros((4, 4, 64)), np.full((4, 4, 64), 1e-30)
    for s, n in enumerate(lengths[:3]):
        at = np.arange(n)
        for j in range(4):
            h = j // 2
            k, v = (sequence_f64(x, d["table"][s], h, n, 32) for x in (K, V))
            pos = d["pos"][d["table"][s][at // 32], h, at % 32]
            want[s, j], bound[s, j] = by_position(k, v, pos, d["q"][s, j], window, 0.125)
    t, n = dev(d["table"]), dev(d["lengths"])
    g.gguf_kv_evict(d["cache"], t, n, 200, window, recent=window)
    assert host(n).tolist() == [min(x, window) for x in lengths]
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), t, n, 200))
    check_bound(got, want, bound, (kind, window))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(TYPES))
def test_windows_count_slots_after_an_eviction(kind):
    rng = np.random.default_rng(61)
    d = make(rng, TYPES[kind], [200, 90, 130], 7, 4, 2, 64, 32, poisoned=False, planes=True)
    planes(d, rng)
    t, n = dev(d["table"]), dev(d["lengths"])
    g.gguf_kv_evict(d["cache"], t, n, 200, 64, recent=8)
    after = dict(d, k=host(d["cache"].k), v=host(d["cache"].v), lengths=host(n))
    for window in (0, 16, 40):
        got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), t, n, 200, window=window))
        want, bound, _ = attend_reference(after, 0.125, window=window)
        check_bound(got, want, bound, (kind, window))
