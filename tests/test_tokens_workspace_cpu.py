"""The workspace of the attention of several new tokens, without a GPU: the size named
for a batch and a bound serves every smaller one."""

import os
import random

import pytest
import torch

import gguf_block_quant_dequant_amd as g
from gguf_block_quant_dequant_amd.build import LIB_PATH
from tests.test_tokens_abi_cpu import cache, extend

pytestmark = [pytest.mark.skipif(not os.path.exists(LIB_PATH), reason="libgguf_qk.so not built"),
              pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="made-up device addresses: only where no GPU is visible")]

F32, BF16 = 0, 30


def named(c, type_, n, rows, heads, max_len, window=0, sinks=0):
    return g.lib().gguf_attn_extend_workspace(c.ref, type_, n, rows, heads, max_len, window, sinks)


def serves(c, have, type_, n, rows, heads, max_len, window=0, sinks=0):
    """Whether a call is let through to the device with this much workspace."""
    st = extend(c, type_=type_, n=n, rows=rows, heads=heads, max_len=max_len, window=window, sinks=sinks, qs=1 << 14,
                os_=1 << 14, q=1 << 44, out=1 << 45, ws=1 << 46, wn=have)
    assert st in (g.ERR_DEVICE, g.ERR_LIMIT), st
    return st == g.ERR_DEVICE


def test_a_size_for_the_greatest_batch_serves_smaller_ones():
    c = cache()
    for type_, large, small in [(F32, (128, 640, 16, 1024), (64, 320, 16, 1024)),    # drafts of fewer sequences
                                (BF16, (1, 2048, 16, 2048), (1, 1024, 16, 2048)),    # a shorter prompt
                                (BF16, (32, 4127, 16, 32768), (31, 31, 16, 32768)),  # the single tokens without it
                                (F32, (64, 64, 16, 131072), (8, 40, 16, 30000)),
                                (BF16, (8, 8192, 16, 8192), (8, 40, 16, 8192))]:
        assert serves(c, named(c, type_, *large), type_, *small), (type_, large, small)


@pytest.mark.parametrize("kind", [1, 30, 8])
def test_the_named_size_grows_with_sequences_rows_and_bound(kind):
    rng = random.Random(kind)

    def size(most):
        return int(most ** rng.random()) if rng.random() < 0.8 else rng.randint(1, 9)
    for _ in range(40):
        hkv = rng.choice([1, 2, 3, 4, 8])
        c = cache(type=kind, page_size=rng.choice([16, 32, 64, 128, 256]), head_dim=rng.choice([64, 96, 128, 192, 256]),
                  n_kv_heads=hkv)
        heads, type_ = hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([F32, BF16])
        if heads * 256 > 1 << 14:
            continue
        window, sinks = rng.choice([0, 0, 1, 300, 5000]), rng.choice([0, 0, 4, 700])
        for _ in range(60):
            n, max_len = size(3000), size(200000)
            rows = n if rng.random() < 0.3 else size(20000)
            have = named(c, type_, n, rows, heads, max_len, window, sinks)
            assert have >= 0
            for _ in range(8):
                a = (rng.randint(1, n) if rng.random() < 0.7 else n, rng.randint(1, rows) if rng.random() < 0.7 else rows)
                b = rng.randint(0, max_len) if rng.random() < 0.7 else max_len
                what = (type_, a, heads, b, window, sinks, (n, rows, max_len))
                assert named(c, type_, *a, heads, b, window, sinks) <= have, what
                assert serves(c, have, type_, *a, heads, b, window, sinks), what


def test_limits_that_the_header_names():
    c = cache()
    # tiles of 16 columns, 4 query heads per kv head: (4 n + 15 n) / 16 <= 65535
    assert named(c, F32, 55188, 55188, 16, 64) == 0 and named(c, F32, 55189, 55189, 16, 64) == g.ERR_LIMIT
    # of 128: (4 n + 127) / 128
    assert named(c, BF16, 1, 65535 * 32, 16, 64) == 0 and named(c, BF16, 1, 65535 * 32 + 1, 16, 64) == g.ERR_LIMIT
    assert named(c, F32, 1, 1 << 20, 16, 64) == g.ERR_LIMIT
    for rows, vocab in (((1 << 23) - 1, 8192), ((1 << 22) - 1, 8193)):
        assert g.gguf_verify_draft_workspace(rows, 4, vocab, True) > 0
        assert g.gguf_verify_draft_workspace(rows + 1, 4, vocab, True) == g.ERR_LIMIT
    assert g.gguf_verify_draft_workspace(8, 65535, 100, True) > 0
    assert g.gguf_verify_draft_workspace(8, 65536, 100, True) == g.ERR_LIMIT
