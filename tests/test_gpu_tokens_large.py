"""The operators over several new tokens where byte offsets pass 32 bits: rows of
queries, outputs and logits far apart, pages of the cache behind the first 4 GiB. What
is computed there equals what the same call computes of a compact copy."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from tests.serving_util import DEV, TYPES, dev
from tests.tokens_util import BF16, make_rows

pytestmark = pytest.mark.gpu

OFFSET = 1 << 32


def say(*a):
    print(*a, flush=True)


def far_rows(x):
    """x's rows spread over more than 4 GiB."""
    es = x.element_size()
    stride = (OFFSET // es // (len(x) - 1) + x.shape[1] + 15) // 16 * 16
    wide = torch.empty(stride * (len(x) - 1) + x.shape[1], dtype=x.dtype, device=x.device)
    rows = wide.as_strided(x.shape, (stride, 1))
    rows.copy_(x)
    assert (len(x) - 1) * stride * es >= OFFSET
    return rows


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_pages_behind_four_gigabytes(kind, bf16):
    rng = np.random.default_rng([31, bf16])
    for rows in ([1, 1], [3, 9], [200, 130]):
        d = make_rows(rng, TYPES[kind], [700, 300], rows, 3, 4, 2, 256, 256, bf16)
        page = d["k"].shape[1]
        base = OFFSET // page + 3
        k, v = (torch.empty((base + d["n_pages"], page), dtype=torch.uint8, device=DEV) for _ in range(2))
        k[base:], v[base:] = dev(d["k"]), dev(d["v"])
        far = g.KvCache(k, v, d["type"], 2, 256, 256)
        say("far pages", kind, rows)
        args = dev(d["lengths"]), 700
        near = g.gguf_attn_extend(d["cache"], d["Q"], dev(d["table"]), *args, row_start=dev(d["starts"]), window=400, sinks=9)
        got = g.gguf_attn_extend(far, d["Q"], dev(d["table"] + base), *args, row_start=dev(d["starts"]), window=400, sinks=9)
        assert torch.isfinite(near.float()).all() and torch.equal(got, near)


@pytest.mark.parametrize("bf16", [False, True])
def test_far_rows_of_queries(bf16):
    rng = np.random.default_rng([32, bf16])
    d = make_rows(rng, BF16, [700, 300], [500, 200], 11, 4, 2, 64, 64, bf16)
    args = dev(d["table"]), dev(d["lengths"]), 700
    near = g.gguf_attn_extend(d["cache"], d["Q"], *args, row_start=dev(d["starts"]))
    out = far_rows(torch.zeros_like(d["Q"]))
    say("far rows")
    g.gguf_attn_extend(d["cache"], far_rows(d["Q"]), *args, row_start=dev(d["starts"]), out=out)
    assert torch.equal(out.contiguous(), near)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 26])
def test_far_rows_of_the_rotation(dim, dtype):
    rng = np.random.default_rng([33, dim])
    n = 4100
    q, k = (dev(rng.standard_normal((n, h * dim)).astype(np.float32)).to(dtype) for h in (3, 1))

    def heads(*x):
        return [t.unflatten(1, (-1, dim)) for t in x]
    rope = dict(freqs=dev(1e-2 ** np.linspace(0, 1, dim // 2)), pos=dev(np.arange(n, dtype=np.int32)))
    near = [x.flatten(1) for x in g.gguf_qk_rope(*heads(q, k), **rope)]
    outs = [far_rows(torch.zeros_like(x)) for x in (q, k)]
    say("far rotation", dim, dtype)
    g.gguf_qk_rope(*heads(far_rows(q), far_rows(k)), **rope, **dict(zip(("q_out", "k_out"), heads(*outs))))
    assert all(torch.equal(o.contiguous(), x) for o, x in zip(outs, near))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [9000, 8999])
def test_far_rows_of_logits(vocab, dtype):
    rng = np.random.default_rng([34, vocab])
    starts = np.array([0, 5, 9, 9, 40], np.int32)
    x, y = (dev(2 * rng.standard_normal((40, vocab)).astype(np.float32)).to(dtype) for _ in range(2))
    args = dict(tokens=dev(rng.integers(0, vocab, 40).astype(np.int32)), uniform=dev(rng.random(40).astype(np.float32)),
                uniform_next=dev(rng.random(4).astype(np.float32)), row_start=dev(starts))
    near = g.gguf_verify_draft(target=x, draft=y, **args)
    say("far logits", vocab, dtype)
    got = g.gguf_verify_draft(target=far_rows(x), draft=far_rows(y), **args)
    assert all(torch.equal(a, b) for a, b in zip(got, near))
