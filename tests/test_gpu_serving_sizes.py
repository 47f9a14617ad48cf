"""Sizes past the loops' first rounds: vocabularies of more splits than a join holds
at once, sequences of more splits than a wave has lanes, evictions of more moves
than the grid has tiles, long prompts, rows past one grid axis."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.formats import f32_to_bf16_bits
from oracle.serving import attend_f64, sequence_f64
from tests.serving_util import DEV, TYPES, U, check_bound, dev, host, make, values
from tests.test_gpu_kv_cache import check_append, check_evict, evict_case

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def check_logprobs(x, tokens, top_k, got):
    """As in the tests of smaller vocabularies; sums over a split's 32 values per
    thread, 64 lanes, 4 waves and n / 8192 splits."""
    lp, ent, ids, top = (host(t) for t in got)
    rel = 2 * (112 + x.shape[1] // 8192) * U
    for r, row in enumerate(x):
        m = row.max()
        lse = np.log(np.exp(row - m).sum())
        order = np.lexsort((np.arange(len(row)), -row))[:top_k]
        assert np.array_equal(ids[r], order), r
        for have, want in ((top[r], row[order] - m - lse), (lp[r], row[tokens[r]] - m - lse)):
            ok = np.isfinite(want)
            assert np.array_equal(have[~ok], want[~ok].astype(np.float32))
            assert (np.abs(have[ok] - want[ok]) <= rel * np.maximum(np.abs(want[ok]), 16)).all(), r
        p = np.exp(row - m - lse)
        h = -(p[p > 0] * (row - m - lse)[p > 0]).sum()
        assert abs(ent[r] - h) <= rel * max(h, 16), r


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab,top_k", [(524289, 64), (1000003, 33), (1048576, 32), (3000001, 1), (600000, 64)])
def test_vocabularies_of_many_splits(vocab, top_k, bf16):
    rng = np.random.default_rng([vocab, 120])
    x = np.stack([2.5 * rng.standard_normal(vocab), np.sort(rng.standard_normal(vocab)),   # the greatest in the last splits
                  np.sort(rng.standard_normal(vocab))[::-1], np.zeros(vocab),
                  np.where(rng.random(vocab) < 0.9999, -np.inf, rng.integers(0, 3, vocab))]).astype(np.float32)
    if bf16:
        x = (f32_to_bf16_bits(x).astype(np.uint32) << 16).view(np.float32)
    tokens = rng.integers(0, vocab, (5, 2))
    t = dev(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16) if bf16 else dev(x)
    say(vocab, top_k, bf16)
    check_logprobs(x.astype(np.float64), tokens, top_k, g.gguf_logprobs(t, dev(tokens.astype(np.int32)), top_k=top_k))


@pytest.mark.parametrize("dim", [64, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_sequences_of_many_splits(kind, dim):
    """Bound as for short sequences, with the roundings of a split's sum (at most 2048
    positions) and of the join over the splits in place of n's."""
    rng = np.random.default_rng([dim, 121])
    n = 70001
    d = make(rng, TYPES[kind], [n], -(-n // 256), 3, 1, dim, 256, planes=True)
    K, V = values(d)
    k, v = (sequence_f64(x, d["table"][0], 0, n, 256) for x in (K, V))
    at = np.arange(n)
    page, slot = d["table"][0][at // 256], at % 256
    scale = dim ** -0.5
    for window in (0, 40000):
        say(kind, dim, window)
        before = host(d["cache"].weight)
        got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), n, track=True,
                                      window=window))
        first = n - window if window else 0
        want, bound, grown, gb = np.zeros((1, 3, dim)), np.zeros((1, 3, dim)), np.zeros(n), np.zeros(n)
        for j in range(3):
            q = d["q"][0, j].astype(np.float64)
            want[0, j], p = attend_f64(q, k[first:], v[first:], scale)
            mag = scale * (np.abs(k[first:]) @ np.abs(q)).max()
            ew = (8 * U + 2.0 ** -22 + 3 * dim * U) * mag + 4 * U + 2.0 ** -22
            rel = 2 * ew + (8 * (2048 + n // 256 + 1) + 128) * U
            bound[0, j] = rel * (p @ np.abs(v[first:]))
            grown[first:] += p
            gb[first:] += rel * p
        check_bound(got, want, bound, (kind, dim, window))
        after = host(d["cache"].weight)[page, 0, slot].astype(np.float64)
        old = before[page, 0, slot].astype(np.float64)
        assert (np.abs(after - old - grown) <= gb + 5 * U * (old + grown) + 1e-36).all()
        assert np.array_equal(after[:first], old[:first])


@pytest.mark.parametrize("kind", list(TYPES))
def test_evictions_of_many_moves(kind):
    # every kept slot lies behind the budget: 70000 moves, past 1024 tiles of 64
    n, budget, ps = 150000, 70000, 256
    d = evict_case(np.random.default_rng(122), kind, [n], ps, hkv=1, ties=False)
    at = np.arange(n)
    d["weight"][d["table"][0][at // ps], 0, at % ps] = at
    d["cache"].weight.copy_(dev(d["weight"]))
    check_evict(d, budget, 0)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("start", [0, 5])
def test_prompts_of_many_tokens(kind, start):
    rng = np.random.default_rng([start, 123])
    n = 9001
    d = make(rng, TYPES[kind], [0, 0], -(-(start + n) // 128), 2, 1, 96, 128, poisoned=False, planes=True)
    k, v = rng.standard_normal((2, n, 96)).astype(np.float32)
    check_append(d, k, v, d["table"], start + np.arange(n), seq=np.zeros(n, int))


@pytest.mark.parametrize("kind", list(TYPES))
def test_evictions_of_long_sequences_with_ties(kind):
    # both ways of holding the keys past the first, of every cache type
    for lengths, budget, recent in (([20000, 17], 6000, 500), ([40000], 30000, 40)):
        check_evict(evict_case(np.random.default_rng([budget, 124]), kind, lengths, 64, hkv=2), budget, recent)


def test_rows_past_one_grid_axis_with_a_join():
    gen = torch.Generator(device=DEV).manual_seed(125)
    x = torch.randn((32771, 9000), generator=gen, device=DEV, dtype=torch.bfloat16)
    tokens = torch.randint(0, 9000, (32771, 2), generator=gen, device=DEV, dtype=torch.int32)
    got = g.gguf_logprobs(x, tokens, top_k=5)
    pick = torch.tensor([0, 1, 32767, 32768, 32770], device=DEV)
    check_logprobs(host(x[pick].double()), host(tokens[pick]), 5, tuple(t[pick] for t in got))
