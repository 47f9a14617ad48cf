"""Pins of the oracle of the serving steps against closed forms and hand examples."""

import math

import numpy as np

from oracle.formats import dequant_q8_0_f64, f32_to_bf16_bits, quantize_q8_0_row
from oracle.serving import (BF16, F16, Q8_0, attend_f64, evict_moves, kv_values_f64, logprobs_f64, sequence_f64)


def test_attend_closed_forms():
    # equal scores: the mean; one score far above: its value
    v = np.arange(12.0).reshape(4, 3)
    out, p = attend_f64(np.zeros(2), np.ones((4, 2)), v, 1.0)
    assert np.allclose(p, 0.25) and np.allclose(out, v.mean(0))
    k = np.array([[0.0], [200.0], [0.0], [0.0]])
    out, p = attend_f64(np.ones(1), k, v, 1.0)
    assert np.allclose(out, v[1], rtol=0, atol=1e-60 + 1e-12)
    # two positions a log-odds of ln 3 apart: 3/4 and 1/4
    out, p = attend_f64(np.ones(1), np.array([[math.log(3.0)], [0.0]]), np.array([[4.0], [8.0]]), 1.0)
    assert np.allclose(p, [0.75, 0.25]) and np.allclose(out, [5.0])
    assert np.array_equal(attend_f64(np.ones(3), np.zeros((0, 3)), np.zeros((0, 3)), 1.0)[0], np.zeros(3))


def test_cache_decode_places_values():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 16, 64)).astype(np.float32)   # [page, head, slot, dim]
    half = x.astype(np.float16)
    assert np.array_equal(kv_values_f64(half.view(np.uint8), F16, 2, 3, 64, 16, False), half.astype(np.float64))
    t = np.ascontiguousarray(np.swapaxes(half, -1, -2))
    assert np.array_equal(kv_values_f64(t.view(np.uint8), F16, 2, 3, 64, 16, True), half.astype(np.float64))
    bits = f32_to_bf16_bits(x)
    assert np.array_equal(kv_values_f64(bits.view(np.uint8), BF16, 2, 3, 64, 16, False),
                          (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64))


def test_cache_decode_q8_0_matches_the_block_format():
    # the same codes and scales as Q8_0 blocks of the rows
    rng = np.random.default_rng(2)
    rows = rng.standard_normal((16, 64)).astype(np.float32)
    blocks = np.frombuffer(b"".join(quantize_q8_0_row(r) for r in rows), np.uint8)
    want = dequant_q8_0_f64(blocks, 16, 64)
    b = blocks.reshape(16, 2, 34)
    codes, scales = b[:, :, 2:].reshape(16, 64), np.ascontiguousarray(b[:, :, :2]).reshape(16, 4)
    k = np.concatenate([codes.reshape(-1), scales.reshape(-1)])
    assert np.array_equal(kv_values_f64(k, Q8_0, 1, 1, 64, 16, False)[0, 0], want)
    v = np.concatenate([np.ascontiguousarray(codes.T).reshape(-1),
                        np.ascontiguousarray(scales.view(np.uint16).T).view(np.uint8).reshape(-1)])
    assert np.array_equal(kv_values_f64(v, Q8_0, 1, 1, 64, 16, True)[0, 0], want)


def test_sequence_follows_the_table():
    pages = np.arange(3 * 1 * 16 * 1, dtype=np.float64).reshape(3, 1, 16, 1)
    got = sequence_f64(pages, [2, 0], 0, 20, 16)[:, 0]
    assert np.array_equal(got, list(range(32, 48)) + list(range(4)))


def test_evict_hand_examples():
    kept, src, dst = evict_moves([5, 1, 3, 2, 9], range(5), 3, 0)
    assert kept.tolist() == [0, 2, 4] and src.tolist() == [4] and dst.tolist() == [1]
    # ties keep the lower slots; the newest token stays whatever its weight
    kept, src, dst = evict_moves([1, 1, 1, 1], range(4), 2, 0)
    assert kept.tolist() == [0, 1] and not len(src)
    kept, src, dst = evict_moves([1, 1, 1, 0], range(4), 2, 1)
    assert kept.tolist() == [0, 3] and src.tolist() == [3] and dst.tolist() == [1]
    # the newest by position, not by slot
    kept, _, _ = evict_moves([0, 1, 1, 1], [7, 0, 1, 2], 2, 1)
    assert kept.tolist() == [0, 1]
    kept, _, _ = evict_moves([0, math.nan, math.inf, 1], range(4), 2, 0)
    assert kept.tolist() == [1, 2]
    assert evict_moves([1, 2], range(2), 2, 0)[1].size == 0


def test_logprobs_closed_forms():
    given, h, ids, top = logprobs_f64(np.zeros(8), [3, -1, 8], 2)
    assert np.allclose(given[0], -math.log(8)) and np.all(np.isneginf(given[1:]))
    assert np.isclose(h, math.log(8)) and ids.tolist() == [0, 1]
    x = np.array([0.0, math.log(3.0), -np.inf])
    given, h, ids, top = logprobs_f64(x, [1, 2], 3)
    assert np.isclose(given[0], math.log(0.75)) and np.isneginf(given[1])
    assert np.isclose(h, -(0.75 * math.log(0.75) + 0.25 * math.log(0.25))) and ids.tolist() == [1, 0, 2]
    # shifted logits have the same probabilities
    r = np.random.default_rng(3).standard_normal(100)
    a, b = logprobs_f64(r, [5], 4), logprobs_f64(r + 50.0, [5], 4)
    assert np.allclose(a[0], b[0]) and np.isclose(a[1], b[1]) and np.array_equal(a[2], b[2])
    assert np.isnan(logprobs_f64([np.nan, 1.0], [1], 1)[1]) and logprobs_f64([1.0, np.nan], [0], 1)[2][0] == 1
