"""The rotation at positions of any size: the angle is the product of a position and an
fp64 frequency, of which nothing that fp32 shows is lost, however many turns it makes.

The reference takes the products in the extended type (64 bits: 2^31 radians to 2^-33)
and is rounded to fp64 at the end; the bound is that of near positions."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from tests.serving_util import DEV, U, dev
from tests.tokens_util import HALF_BF16, as_f64, as_type

pytestmark = pytest.mark.gpu

FAR = [0, 1, -1, 131071, 2 ** 24 + 1, 987654321, -(2 ** 30) - 5, 2 ** 31 - 1, 2 ** 31 - 2, -(2 ** 31), 2 ** 30 + 7]


@pytest.mark.skipif(np.finfo(np.longdouble).nmant < 63, reason="no extended type")
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("pad", [0, 1])   # 1: rows that are not 16-byte aligned
@pytest.mark.parametrize("bf16", [False, True])
def test_far_positions(bf16, pad, halves):
    rng = np.random.default_rng([11, bf16, pad, halves])
    n, heads, dim = len(FAR), 3, 64
    freqs = np.concatenate([[1.0, 0.999, 2.0 / 3.0], 3.0 * rng.random(29)])
    buf, x = as_type(rng.standard_normal((n, heads * dim + pad)), bf16)
    x = x[:, :heads * dim].reshape(n, heads, dim)
    q = buf[:, :heads * dim].unflatten(1, (heads, dim))
    got = as_f64(g.gguf_qk_rope(q, None, dev(np.array(FAR, np.int32)), torch.tensor(freqs, device=DEV), halves=halves)[0])
    angle = np.array(FAR, np.longdouble)[:, None] * freqs.astype(np.longdouble)
    c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    a, b = (slice(0, 32), slice(32, 64)) if halves else (slice(0, None, 2), slice(1, None, 2))
    want, bound = np.empty_like(x), np.empty_like(x)
    want[..., a], want[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    # the fraction of a turn rounds by 2^-26 turns (1.6 U), the functions by 2 ulp (4 U), products and sum by 2 U
    bound[..., a] = bound[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * (8 * U + 2.0 ** -33) + 1e-37
    if bf16:
        bound += HALF_BF16 * (np.abs(want) + bound)
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), (float(over.max()), np.argwhere(over > 0)[:4])
