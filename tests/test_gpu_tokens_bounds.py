"""The bounds that the header names for draws from max(p - q, 0) where the draft is close
to its target, and for queries whose elements lie far below their row's greatest."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.serving import attend_f64, sequence_f64
from tests.serving_util import F16, Q8_0, U, dev, host, values
from tests.tokens_util import HALF_BF16, HALF_F16, as_f64, as_type, extend, make_rows

pytestmark = pytest.mark.gpu


@pytest.mark.skipif(np.finfo(np.longdouble).nmant < 63, reason="no extended type")
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("noise", [1e-1, 1e-3, 1e-6])
def test_draws_from_what_a_close_draft_leaves(noise, bf16):
    """With R the whole of max(p - q, 0) a draw is the lowest i whose running sum exceeds
    uniform_next R, but for sums within 1e-12 (of the probabilities' whole, 1): both weights
    are off by 2^-43 and a rounding, and their sums by less."""
    rng = np.random.default_rng([51, bf16, int(-np.log10(noise))])
    vocab, seqs = 5000, 64
    x = 2.0 * rng.standard_normal((2 * seqs, vocab))
    tx, x = as_type(x, bf16)
    y = x + noise * rng.standard_normal(x.shape)
    if bf16:   # a few logits a step apart, the others alike
        y = np.where(rng.random(x.shape) < noise, x * (1 + 2.0 ** -7), x)
    ty, y = as_type(y, bf16)
    p, q = (np.exp((z - z.max(1, keepdims=True)).astype(np.longdouble)) for z in (x, y))
    p, q = p / p.sum(1, keepdims=True), q / q.sum(1, keepdims=True)
    rest = np.maximum(p - q, 0)[0::2]
    # drafts that are refused: of the least p / q, beside a number just below one
    tokens = np.zeros(2 * seqs, np.int32)
    tokens[0::2] = (p / q)[0::2].argmin(1)
    u = np.full(2 * seqs, 1.0 - 2.0 ** -24, np.float32)
    un = rng.random(seqs).astype(np.float32)
    starts = 2 * np.arange(seqs + 1, dtype=np.int32)
    r = g.gguf_verify_draft(tx, dev(tokens), dev(u), dev(un), dev(starts), draft=ty)
    taken, accepted = host(r.next_tokens), host(r.accepted)
    ratio = (p / q)[0::2].min(1)
    refused = ratio < 1 - 2.0 ** -20
    assert refused.sum() > (seqs // 2 if noise > 1e-6 or not bf16 else -1) and (accepted[refused] == 0).all()
    run = np.cumsum(rest, 1)
    goal = un.astype(np.longdouble) * run[:, -1]
    for s in np.flatnonzero(refused):
        i = taken[s]
        assert rest[s, i] > 0, (s, i)
        assert run[s, i] > goal[s] - 1e-12 and run[s, i] - rest[s, i] <= goal[s] + 1e-12, (s, i, float(run[s, -1]))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("type_id", [F16, Q8_0])
def test_queries_far_below_their_greatest(type_id, dim):
    """BF16 rows over F16 and Q8_0 caches where many rows run: elements below 2^-26 of the
    row's greatest are within 2^-34 of it, others exact. The greatest meets keys of zero, so
    that the scores are the small elements' alone."""
    rng = np.random.default_rng([52, dim])
    d = make_rows(rng, type_id, [200], [64], 4, 2, 1, dim, 64, True)
    raw = d["k"].reshape(d["n_pages"], -1).copy()
    if type_id == F16:   # the first dim of every key
        raw.view(np.uint16).reshape(d["n_pages"], 64, dim)[:, :, 0] = 0
    else:
        raw[:, :64 * dim].reshape(d["n_pages"], 64, dim)[:, :, 0] = 0
    d["k"] = raw
    d["cache"] = g.KvCache(dev(raw), dev(d["v"]), type_id, 1, dim, 64)
    q = rng.standard_normal((64, 2, dim)) * 2.0 ** -rng.integers(18, 36, (64, 2, 1))
    q[:, :, 0] = rng.choice([-1.0, 1.0], (64, 2)) * rng.uniform(0.5, 2, (64, 2))
    d["Q"], d["q"] = as_type(q.reshape(64, -1), True)
    K, V = values(d)
    scale = 2.0 ** 24
    got = as_f64(extend(d, scale=scale)).reshape(64, 2, dim)
    assert np.isfinite(got).all()
    for j in range(0, 64, 7):
        see = np.arange(200 - 64 + j + 1)
        k, v = (sequence_f64(x, d["table"][0], 0, 200, 64)[see] for x in (K, V))
        for h in range(2):
            x = d["q"][j].reshape(2, dim)[h]
            o, p = attend_f64(x, k, v, scale)
            mag = scale * (np.abs(k) @ np.abs(x)).max()
            kq = HALF_F16 if type_id == Q8_0 else 0.0
            es = (4 * U + kq + 3 * dim * U) * mag + scale * 2.0 ** -34 * np.abs(x).max() * np.abs(k).sum(1).max()
            ew = es + 4 * U * mag + 4 * U
            bound = (2 * ew + 2 * HALF_F16 + (8 * len(p) + 128) * U) * (p @ np.abs(v)) + 2.0 ** -25 * p.max() * np.abs(v).sum(0)
            bound += HALF_BF16 * (np.abs(o) + bound)
            assert (np.abs(got[j, h] - o) <= bound).all(), (j, h, float((np.abs(got[j, h] - o) - bound).max()))
