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


def test_workspace_serves_smaller_batches_bounds_and_any_window():
    """The bytes named for a batch and a bound are enough for every call with at most
    as many sequences and at most that bound."""
    rng = np.random.default_rng(70)
    head_dims = {16: 64, 64: 128, 256: 256}
    for ps, dim in head_dims.items():
        for kind in (g.TENSOR_BF16, g.TYPE_Q8_0):
            for heads, hkv in ((16, 4), (4, 4), (40, 1)):
                c = abi.cache(type=kind, page_size=ps, head_dim=dim, n_kv_heads=hkv)
                for seqs, max_len in ((5, 32768), (9, 32768), (64, 1000), (33, 300), (300, 8192), (3, 70000)):
                    for track in (0, 1):
                        need = g.lib().gguf_attn_decode_workspace(c.ref, seqs, heads, max_len, track)
                        assert need >= 0
                        last = 0
                        for n in sorted({1, 2, 3, seqs // 2, seqs - 1, seqs}):
                            own = g.lib().gguf_attn_decode_workspace(c.ref, n, heads, max_len, track)
                            assert last <= own <= need, (ps, kind, heads, seqs, max_len, track, n)
                            last = own
                            for m in {max_len, max_len // 2, 513, 512, 257, 64, int(rng.integers(1, max_len))}:
                                if m > max_len:
                                    continue
                                for window in (0, 1, 300, int(rng.integers(1, m + 1))):
                                    got = abi.attend(c, n=n, heads=heads, max_len=m, window=window, track=track,
                                                     wn=need, qs=heads * dim, os_=heads * dim, table=1 << 56,
                                                     lengths=1 << 57, q=1 << 58, out=1 << 59, ws=1 << 60)
                                    assert got == g.ERR_DEVICE, (ps, kind, heads, seqs, max_len, track, n, m, window)
