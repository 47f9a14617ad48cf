"""Attention at the edges of its numbers: queries up to fp32's greatest values, V's
values and scales over fp16's whole range against the weights."""

import numpy as np
import pytest

import gguf_block_quant_dequant_amd as g
from oracle.formats import f32_to_bf16_bits
from oracle.serving import attend_f64
from tests.serving_util import DEV, TYPES, U, attend_reference, check_bound, dev, host, make, values
from tests.test_gpu_kv_cache import views

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [100, 112, 116, 119, 122])
@pytest.mark.parametrize("kind", list(TYPES))
def test_queries_near_the_top_of_fp32(kind, exponent):
    """Scores of 1e27 and more: finite, and so far apart that the greatest takes all
    the weight. The output is then its value: the weight is exactly 1, its parts
    add up to it, the value is exact (Q8_0: code times scale, one rounding)."""
    rng = np.random.default_rng([exponent, 80])
    d = make(rng, TYPES[kind], [1, 40, 150, 700], 11, 4, 2, 64, 64, scale=2.0 ** -10)
    d["q"] = (d["q"] * np.float32(2.0 ** exponent)).astype(np.float32)
    assert np.isfinite(d["q"]).all()
    K, V = values(d)
    want = np.zeros((4, 4, 64))
    for s, n in enumerate(d["lengths"]):
        at = np.arange(n)
        page, slot = d["table"][s][at // 64], at % 64
        for j in range(4):
            scores = K[page, j // 2, slot] @ d["q"][s, j].astype(np.float64)
            assert np.abs(scores).max() * 1.45 < 3.4e38
            order = np.argsort(-scores)
            if n > 1:
                # far past the scores' error (64 products of 2^-22 and 3 * 64 roundings)
                mag = (np.abs(K[page, j // 2, slot]) @ np.abs(d["q"][s, j].astype(np.float64))).max()
                assert scores[order[0]] - scores[order[1]] > 2.0 ** -14 * mag
            want[s, j] = V[page, j // 2, slot][order[0]]
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 700, scale=1.0))
    check_bound(got, want, 4 * U * np.abs(want), (kind, exponent))


def against_the_weights(d, low, high):
    """V of the first sequence from 2^low, where a head's weight is greatest, to
    2^high where it is least (F16, BF16: values; Q8_0: scales, codes as they are)."""
    K, _ = values(d)
    n, ps = int(d["lengths"][0]), d["ps"]
    at = np.arange(n)
    page, slot = d["table"][0][at // ps], at % ps
    parts = views(d["v"], d["type"], d["n_pages"], d["hkv"], d["dim"], ps, True)
    for h in range(d["hkv"]):
        scores = K[page, h, slot] @ d["q"][0, h * d["heads"] // d["hkv"]].astype(np.float64)
        rank = np.empty(n)
        rank[np.argsort(-scores)] = np.arange(n)
        size = np.exp2(low + (high - low) * rank / (n - 1))
        if d["type"] == TYPES["q8_0"]:
            parts[1][page, h, slot] = size[:, None].astype(np.float16).view(np.uint16)
        else:
            sign = np.where(np.random.default_rng(h).random((n, d["dim"])) < 0.5, -1.0, 1.0)
            x = (size[:, None] * sign).astype(np.float32)
            parts[0][page, h, slot] = (x.astype(np.float16).view(np.uint16) if d["type"] == TYPES["f16"]
                                       else f32_to_bf16_bits(x))
    d["cache"].v.copy_(dev(d["v"]).view(d["cache"].v.shape))


def floors(d, scale):
    """What the parts of the weights may be off by beside their 22 bits (which the
    reference's bound counts): per output 2^-39 of the greatest weight times every
    |v| (F16); for Q8_0 the greatest weight times every |code| times the greatest of
    2^-39 of the block's greatest scale, 2^-54 of the head's, and 2^-54."""
    K, V = values(d)
    n, ps, group = int(d["lengths"][0]), d["ps"], d["heads"] // d["hkv"]
    at = np.arange(n)
    page, slot = d["table"][0][at // ps], at % ps
    out = np.zeros((1, d["heads"], d["dim"]))
    if d["type"] == TYPES["bf16"]:
        return out
    parts = views(d["v"], d["type"], d["n_pages"], d["hkv"], d["dim"], ps, True)
    for j in range(d["heads"]):
        h = j // group
        _, p = attend_f64(d["q"][0, j], K[page, h, slot], V[page, h, slot], scale)
        if d["type"] == TYPES["f16"]:
            out[0, j] = p.max() * 2.0 ** -39 * np.abs(V[page, h, slot]).sum(0)
        else:
            scales = np.abs(parts[1][page, h, slot].view(np.float16).astype(np.float64))
            unit = np.maximum(2.0 ** -39 * scales.max(0), 2.0 ** -54 * max(1.0, scales.max()))
            codes = np.abs(parts[0][page, h, slot].view(np.int8).astype(np.float64))
            out[0, j] = p.max() * codes.sum(0) * np.repeat(unit, 32)
    return out


@pytest.mark.parametrize("low,high", [(-24, 15), (-14, 15), (-24, -4), (-5, 5)])
@pytest.mark.parametrize("n", [24, 300])
@pytest.mark.parametrize("kind", list(TYPES))
def test_values_large_where_weights_are_small(kind, n, low, high):
    rng = np.random.default_rng([n, 81])
    d = make(rng, TYPES[kind], [n], 5, 4, 2, 64, 64, poisoned=False)
    against_the_weights(d, low, high)
    want, bound, _ = attend_reference(d, 0.125)
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), n))
    check_bound(got, want, bound + floors(d, 0.125), (kind, n, low, high))


@pytest.mark.parametrize("small,large", [(1e-3, 3e3), (1e-6, 6e4), (2.0 ** -24, 6e4), (1e-6, 1e-6)])
def test_q8_0_small_blocks_beside_large_ones(small, large):
    rng = np.random.default_rng(82)
    d = make(rng, TYPES["q8_0"], [40], 1, 4, 2, 128, 64, poisoned=False)
    parts = views(d["v"], d["type"], d["n_pages"], 2, 128, 64, True)
    parts[1][..., :2] = np.float16(small).view(np.uint16)
    parts[1][..., 2:] = np.float16(large).view(np.uint16)
    d["cache"].v.copy_(dev(d["v"]).view(d["cache"].v.shape))
    d["q"] *= np.float32(0.25)
    want, bound, _ = attend_reference(d, 0.0884)
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 40, scale=0.0884))
    check_bound(got, want, bound + floors(d, 0.0884), (small, large))
