"""Log probabilities, entropy and top alternatives against the fp64 oracle: odd
vocabularies, strides and alignments, ties, ruled-out tokens, special values."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.formats import f32_to_bf16_bits
from oracle.serving import logprobs_f64
from tests.serving_util import DEV, U, dev, host

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def check(x, tokens, top_k, got, what):
    """x: fp64 values of the logits. The log probabilities: log L and x - max
    round by U of their magnitude each, L carries the exponentials' error (an
    argument rounded by 2 U |d| with weight e^d: at most 2 U, the function 2 U)
    and the sums' (32 per thread, 64 lanes by halves, 4 waves, the splits: at
    most 32 + 8 + 4 + 64 roundings)."""
    lp, ent, ids, top = (None if t is None else host(t) for t in got)
    for r in range(len(x)):
        given, h, order, best = logprobs_f64(x[r], tokens[r] if tokens is not None else [], top_k)
        if tokens is not None:
            close(lp[r], given, what)
        close(ent[r:r + 1], np.array([h]), what, entropy=True)
        if top_k:
            assert np.array_equal(ids[r], order), (what, r, ids[r], order)
            close(top[r], best, what)


def close(got, want, what, entropy=False):
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, got, want)
    assert np.array_equal(np.isinf(got), np.isinf(want)) and np.array_equal(got[np.isinf(got)], want[np.isinf(want)])
    ok = np.isfinite(want)
    # the entropy: log L - T / L, T's terms rounded three times more
    rel = (112 + (112 if entropy else 0)) * U
    assert (np.abs(got[ok] - want[ok]) <= rel * np.maximum(np.abs(want[ok]), 16.0)).all(), (what, got, want)


def call(x, tokens, top_k, bf16, **kw):
    t = dev(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16) if bf16 else dev(x)
    return g.gguf_logprobs(t, None if tokens is None else dev(tokens.astype(np.int32)), top_k=top_k, **kw)


def logits(rng, n, vocab, bf16):
    x = (2.5 * rng.standard_normal((n, vocab))).astype(np.float32)
    return (f32_to_bf16_bits(x).astype(np.uint32) << 16).view(np.float32) if bf16 else x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 64, 65, 255, 511, 700, 997, 1025, 4095, 8185, 8189, 8192, 8193, 16384,
                                   16391, 32000, 50257, 128256])
def test_vocabularies(vocab, bf16):
    rng = np.random.default_rng([vocab, bf16])
    x = logits(rng, 3, vocab, bf16)
    tokens = rng.integers(0, vocab, (3, 4))
    tokens[1, 2], tokens[2, 0], tokens[2, 1] = -1, vocab, 2 ** 31 - 1
    for k in sorted({0, 1, min(5, vocab), min(20, vocab), min(64, vocab)}):
        say("logprobs", vocab, bf16, k)
        check(x.astype(np.float64), tokens, k, call(x, tokens, k, bf16), (vocab, k))


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_apart_and_unaligned(bf16):
    rng = np.random.default_rng(2)
    for vocab, stride, offset in ((1000, 1001, 0), (8200, 8211, 3), (501, 517, 1), (20001, 20001, 5)):
        n = 5
        x = logits(rng, 1, n * stride + offset + 8, bf16)[0]
        flat = dev(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16) if bf16 else dev(x)
        rows = torch.as_strided(flat, (n, vocab), (stride, 1), offset)
        want = np.lib.stride_tricks.as_strided(x[offset:], (n, vocab), (stride * 4, 4)).astype(np.float64)
        tokens = rng.integers(0, vocab, (n, 1))
        check(want, tokens, 10, g.gguf_logprobs(rows, dev(tokens.astype(np.int32)), top_k=10), (vocab, stride, offset))


@pytest.mark.parametrize("vocab", [300, 5000, 20000])
def test_ties_and_ruled_out_tokens(vocab):
    rng = np.random.default_rng([vocab, 3])
    rows = [np.zeros(vocab), np.full(vocab, -7.5), rng.integers(0, 3, vocab).astype(float),
            np.where(rng.random(vocab) < 0.99, -np.inf, 1.0), np.where(np.arange(vocab) == vocab - 1, 0.0, -np.inf),
            np.where(np.arange(vocab) % 2, 0.0, -0.0), -np.abs(rng.standard_normal(vocab)) * 1e30,
            np.sort(rng.standard_normal(vocab)), np.sort(rng.standard_normal(vocab))[::-1],
            np.where(np.arange(vocab) < 40, 1.0, -np.inf), np.full(vocab, np.finfo(np.float32).min)]
    x = np.stack(rows).astype(np.float32)
    tokens = rng.integers(0, vocab, (len(rows), 3))
    for k in (1, 8, 33, 64):
        check(x.astype(np.float64), tokens, k, call(x, tokens, k, False), (vocab, k))


@pytest.mark.parametrize("vocab", [100, 30000])
def test_nan_infinity_and_empty_rows(vocab):
    rng = np.random.default_rng([vocab, 4])
    x = rng.standard_normal((5, vocab)).astype(np.float32)
    x[0, 37] = np.nan
    x[1, [5, 60]] = np.inf
    x[2] = -np.inf                      # every token ruled out
    x[3] = np.nan
    x[4, :50] = -np.inf
    tokens = np.tile(np.array([37, 5, -1]), (5, 1))
    r = call(x, tokens, 4, False)
    lp, ent, ids, top = (host(t) for t in r)
    for row in (0, 1, 2, 3):
        assert np.isnan(lp[row, :2]).all() and np.isnan(ent[row]) and np.isnan(top[row]).all()
        assert np.isneginf(lp[row, 2])
    assert ids[0, 0] == 37 and ids[1, :2].tolist() == [5, 60] and ids[2].tolist() == [0, 1, 2, 3]
    assert ids[3].tolist() == [0, 1, 2, 3]
    check(x[4:].astype(np.float64), tokens[4:], 4, tuple(t[4:] for t in r), "ruled out")


def test_many_rows_one_row_and_parts():
    rng = np.random.default_rng(5)
    x = logits(rng, 33000, 40, False)    # rows past one grid axis
    tokens = rng.integers(0, 40, (33000, 1))
    r = call(x, tokens, 2, False)
    pick = [0, 1, 32767, 32768, 32999]
    check(x[pick].astype(np.float64), tokens[pick], 2, tuple(t[pick] for t in r), "rows")
    one = call(x[7], tokens[7], 3, False)
    assert one.token_logprobs.shape == (1, 1) and one.top_ids.shape == (1, 3)
    check(x[7:8].astype(np.float64), tokens[7:8], 3, one, "one")
    part = call(x[:3], None, 0, False)
    assert part.token_logprobs is None and part.top_ids is None and part.entropy.shape == (3,)
    none = g.gguf_logprobs(torch.empty((0, 40), device=DEV), torch.empty((0, 1), dtype=torch.int32, device=DEV), top_k=2)
    assert none.entropy.shape == (0,)


def test_streams_graph_and_refusals():
    rng = np.random.default_rng(6)
    x = logits(rng, 4, 40000, True)
    tokens = rng.integers(0, 40000, (4, 2))
    t = dev(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16)
    tk = dev(tokens.astype(np.int32))
    torch.cuda.synchronize()
    first = [host(y) for y in g.gguf_logprobs(t, tk, top_k=20)]
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        outs += [g.gguf_logprobs(t, tk, top_k=20, stream=s) for s in streams]
    torch.cuda.synchronize()
    for o in outs:   # the same bits on every stream and run
        assert all(np.array_equal(host(a).view(np.uint8), b.view(np.uint8)) for a, b in zip(o, first))
    ws = torch.empty(g.gguf_logprobs_workspace(4, 40000, 20), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = g.gguf_logprobs(t, tk, top_k=20, workspace=ws)
    for seed in range(3):
        x = logits(np.random.default_rng(100 + seed), 4, 40000, True)
        t.copy_(dev(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16))
        for y in r:
            y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        check(x.astype(np.float64), tokens, 20, r, seed)
    for bad in (dict(top_k=65), dict(top_k=-1)):
        with pytest.raises((g.GgufQkArgumentError, RuntimeError)):
            g.gguf_logprobs(t, tk, **bad)
    with pytest.raises(g.GgufQkArgumentError):
        g.gguf_logprobs(t, tk, top_k=4, workspace=ws[:64])
    with pytest.raises(ValueError):
        g.gguf_logprobs(t.half(), tk)
    with pytest.raises(ValueError):
        g.gguf_logprobs(t.t(), tk)
    with pytest.raises(ValueError):
        g.gguf_logprobs(t, tk[:3])
    with pytest.raises(ValueError):
        g.gguf_logprobs(t, tk.long())
