"""Shapes of the token lists that gguf_logprobs takes."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from tests.serving_util import DEV, dev, host

pytestmark = pytest.mark.gpu


def test_token_shapes():
    rng = np.random.default_rng(110)
    x = dev(rng.standard_normal((4, 100)).astype(np.float32))
    t = dev(rng.integers(0, 100, (4, 2)).astype(np.int32))
    want = host(g.gguf_logprobs(x, t).token_logprobs)
    assert want.shape == (4, 2)
    one = g.gguf_logprobs(x, t[:, 0].contiguous()).token_logprobs   # a token per row
    assert np.array_equal(host(one), want[:, :1])
    row = g.gguf_logprobs(x[1], t[1]).token_logprobs                 # tokens of the one row
    assert np.array_equal(host(row), want[1:2])
    assert g.gguf_logprobs(x, t[:, :0].contiguous()).token_logprobs is None
    # lists that are neither: the same tokens for every row, a flat list, more axes
    for bad in (t.view(8), t[0], t.view(2, 4), t.view(4, 2, 1), t.view(4, 1, 2), t.view(1, 4, 2),
                torch.zeros((), dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError):
            g.gguf_logprobs(x, bad)
