"""Attention at the edges of its numbers: queries up to fp32's greatest values."""

import numpy as np
import pytest

import gguf_block_quant_dequant_amd as g
from tests.serving_util import DEV, TYPES, U, attend_reference, check_bound, dev, host, make, values

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
