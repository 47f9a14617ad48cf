"""Ranges of the attention's arguments at their edges, without a GPU: a call that
passes validation ends at the device check."""

import numpy as np
import pytest

import gguf_block_quant_dequant_amd as g
from tests import test_kv_abi_cpu as abi

pytestmark = abi.pytestmark


def test_scale_up_to_the_type_s_range():
    # the kernels take scale * log2(e): finite up to 2.358e38
    log2e = np.float32(1.44269504)
    c = abi.cache()
    top = np.float32(np.finfo(np.float32).max) / log2e
    inside, outside = np.nextafter(top, np.float32(0)), np.float32(2.36e38)
    with np.errstate(over="ignore"):
        assert np.isfinite(inside * log2e) and np.isinf(outside * log2e)
    for sign in (1, -1):
        for scale in (0.0, 1e-45, 1.0, float(inside)):
            assert abi.attend(c, scale=sign * scale) == g.ERR_DEVICE, scale
        for scale in (float(outside), 2.9e38, 3.0e38, 3.4e38, float("inf")):
            assert abi.attend(c, scale=sign * scale) == g.ERR_SHAPE, scale
