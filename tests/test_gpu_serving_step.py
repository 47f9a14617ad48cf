"""The serving operators in one loop with the products around them, as a decode
step uses them: q, k, v of three sequences (one multi-matrix product), append,
attention with tracked weights, output projection, head, log probabilities, and
eviction at the budget; then the step as one captured graph. Every stage against
the fp64 oracle fed with the stage's own inputs."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
import oracle
import synth
from oracle.serving import BF16, F16, Q8_0, attend_f64, evict_moves, kv_values_f64, logprobs_f64, sequence_f64
from tests.serving_util import DEV, dev, host

pytestmark = pytest.mark.gpu

SEQS, HEADS, KV_HEADS, DIM, PAGE, PAGES, HIDDEN, VOCAB = 3, 8, 2, 64, 16, 4, 512, 1000
BUDGET, RECENT = 40, 6


def say(*a):
    print(*a, flush=True)


def model(rng):
    rows = {"q": HEADS * DIM, "k": KV_HEADS * DIM, "v": KV_HEADS * DIM, "o": HIDDEN, "head": VOCAB}
    raw = {n: synth.q4_k_weights(rng, r, HIDDEN) for n, r in rows.items()}
    return {n: dev(w) for n, w in raw.items()}, {n: oracle.dequant_q4_k_f32(raw[n], r, HIDDEN).astype(np.float64)
                                                 for n, r in rows.items()}


def close(got, want, tol, what):
    e, ok = oracle.floored_rel_err(got, want)
    assert ok and e <= tol, (what, e)


@pytest.mark.parametrize("kind", [F16, BF16, Q8_0])
def test_decode_loop_with_eviction(kind):
    rng = synth.rng_for(51, kind, 0)
    W, W64 = model(rng)
    n_pages = SEQS * PAGES
    cache = g.KvCache.empty(kind, n_pages, KV_HEADS, DIM, PAGE, device=DEV, planes=True)
    table = rng.permutation(n_pages).astype(np.int32).reshape(SEQS, PAGES)
    T = dev(table)
    lengths = torch.zeros(SEQS, dtype=torch.int32, device=DEV)
    max_len = PAGES * PAGE
    evicted = 0
    for step in range(60):
        say("step", step)
        x = (0.05 * rng.standard_normal((SEQS, HIDDEN))).astype(np.float32)
        q, k, v = g.gguf_qmatmul_f32_q4_k_multi([W["q"], W["k"], W["v"]], dev(x))
        close(host(k), x.astype(np.float64) @ W64["k"].T, 1e-3, "k")
        # sequence 2 idles at first: its token is a padding row
        slot = lengths.clone()
        if step < 5:
            slot[2] = -1
        pos = torch.full((SEQS,), step, dtype=torch.int32, device=DEV)
        g.gguf_kv_append(cache, k, v, T, slot, pos=pos)
        lengths += (slot >= 0).int()
        n = host(lengths)
        before = host(cache.weight).astype(np.float64)
        q = q / q.square().mean().sqrt()
        o = g.gguf_attn_decode(cache, q, T, lengths, max_len, track=True)
        vals = [kv_values_f64(host(t), kind, n_pages, KV_HEADS, DIM, PAGE, tr)
                for t, tr in ((cache.k, False), (cache.v, True))]
        want, qh = np.zeros((SEQS, HEADS, DIM)), host(q).reshape(SEQS, HEADS, DIM)
        for s in range(SEQS):
            at = np.arange(n[s])
            for h in range(HEADS):
                kk, vv = (sequence_f64(p, table[s], h // (HEADS // KV_HEADS), n[s], PAGE) for p in vals)
                want[s, h], p = attend_f64(qh[s, h], kk, vv, DIM ** -0.5)
                before[table[s][at // PAGE], h // (HEADS // KV_HEADS), at % PAGE] += p
        close(host(o), want.reshape(SEQS, -1), 1e-4, "attention")
        assert np.allclose(host(cache.weight), before, rtol=1e-4, atol=1e-5)
        y = g.gguf_qmatmul_f32_q4_k(W["o"], o)
        close(host(y), host(o).astype(np.float64) @ W64["o"].T, 1e-3, "output projection")
        logits = g.gguf_qmatmul_f32_q4_k(W["head"], (y / y.square().mean().sqrt() * 0.05).contiguous())
        tokens = dev(rng.integers(0, VOCAB, (SEQS, 1)).astype(np.int32))
        r = g.gguf_logprobs(logits, tokens, top_k=5)
        L = host(logits).astype(np.float64)
        for s in range(SEQS):
            given, ent, ids, best = logprobs_f64(L[s], host(tokens)[s], 5)
            assert np.allclose(host(r.token_logprobs)[s], given, rtol=1e-5, atol=1e-4)
            assert np.allclose(host(r.entropy)[s], ent, rtol=1e-5, atol=1e-4)
            assert np.array_equal(host(r.top_ids)[s], ids) and np.allclose(host(r.top_logprobs)[s], best, atol=1e-4)
        # eviction: the kept positions are the oracle's
        w, ps = host(cache.weight), host(cache.pos)
        expect = {}
        for s in range(SEQS):
            at = np.arange(n[s])
            for h in range(KV_HEADS):
                page, i = table[s][at // PAGE], at % PAGE
                kept, src, _ = evict_moves(w[page, h, i], ps[page, h, i], BUDGET, RECENT)
                expect[s, h] = sorted(ps[page, h, i][kept].tolist())
                evicted += len(src) > 0
        g.gguf_kv_evict(cache, T, lengths, max_len, BUDGET, recent=RECENT)
        n, ps = host(lengths), host(cache.pos)
        for (s, h), want_pos in expect.items():
            at = np.arange(n[s])
            assert sorted(ps[table[s][at // PAGE], h, at % PAGE].tolist()) == want_pos
        assert (n <= BUDGET).all()
    assert evicted > 10 and n.tolist() == [40, 40, 40]


def test_captured_step_replays_like_the_eager_one():
    rng = synth.rng_for(52, 0, 0)
    W, _ = model(rng)
    n_pages = SEQS * PAGES
    T = dev(rng.permutation(n_pages).astype(np.int32).reshape(SEQS, PAGES))
    x = torch.zeros((SEQS, HIDDEN), device=DEV)
    tokens = torch.zeros((SEQS, 1), dtype=torch.int32, device=DEV)
    max_len = PAGES * PAGE

    def fresh():
        return (g.KvCache.empty(F16, n_pages, KV_HEADS, DIM, PAGE, device=DEV, planes=True),
                torch.zeros(SEQS, dtype=torch.int32, device=DEV), torch.zeros(SEQS, dtype=torch.int32, device=DEV))

    def step(cache, lengths, pos):
        q, k, v = g.gguf_qmatmul_f32_q4_k_multi([W["q"], W["k"], W["v"]], x)
        g.gguf_kv_append(cache, k, v, T, lengths, pos=pos)
        lengths += 1
        pos += 1
        o = g.gguf_attn_decode(cache, q, T, lengths, max_len, track=True, scale=0.01)
        logits = g.gguf_qmatmul_f32_q4_k(W["head"], g.gguf_qmatmul_f32_q4_k(W["o"], o))
        r = g.gguf_logprobs(logits, tokens, top_k=3)
        g.gguf_kv_evict(cache, T, lengths, max_len, BUDGET, recent=RECENT)
        return o, r

    eager, graphed = fresh(), fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # warm the stream's scratch slot outside the capture
        step(*fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go, gr = step(*graphed)
    for i in range(50):
        x.copy_(dev((0.05 * rng.standard_normal((SEQS, HIDDEN))).astype(np.float32)))
        tokens.copy_(dev(rng.integers(0, VOCAB, (SEQS, 1)).astype(np.int32)))
        eo, er = step(*eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(eo), host(go)), i
        for a, b in zip(er, gr):
            assert np.array_equal(host(a), host(b)), i
        for a, b in zip((eager[0].k, eager[0].v, eager[0].weight, eager[0].pos, eager[1]),
                        (graphed[0].k, graphed[0].v, graphed[0].weight, graphed[0].pos, graphed[1])):
            assert np.array_equal(host(a), host(b)), i
    g.gguf_qk_stream_release(side)
    g.gguf_qk_stream_release()
