"""The operators over several new tokens as a serving program runs them: a prompt
(bf16 products, norms and rotation, append, attention), then drafted tokens of the
same sequences in fp32 (small-batch products, norms and rotation, append, attention,
head, verification), the cache cut back to what was accepted; then that step as one
captured graph. Every stage against the fp64 oracle fed with the stage's own inputs."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
import oracle
import synth
from oracle.formats import f32_to_bf16_bits
from oracle.serving import BF16, F16, Q8_0, attend_f64, kv_values_f64, sequence_f64
from oracle.tokens import rope_f64, verify_f64, visible_slots
from tests.serving_util import DEV, dev, host
from tests.tokens_util import as_f64

pytestmark = pytest.mark.gpu

SEQS, HEADS, KV_HEADS, DIM, PAGE, PAGES, HIDDEN, VOCAB = 3, 8, 2, 64, 16, 8, 512, 1000
WINDOW, SINKS, DRAFTS = 40, 4, 4
PROMPTS = [70, 33, 1]


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


def check_attention(o, q, cache, kind, table, lengths, rows, tol):
    K, V = (kv_values_f64(host(t), kind, cache.n_pages, KV_HEADS, DIM, PAGE, tr) for t, tr in ((cache.k, False), (cache.v, True)))
    want, r = np.zeros((sum(rows), HEADS, DIM)), 0
    for s, m in enumerate(rows):
        for j in range(m):
            see = visible_slots(lengths[s], m, j, WINDOW, SINKS)
            for h in range(HEADS):
                k, v = (sequence_f64(x, table[s], h // (HEADS // KV_HEADS), lengths[s], PAGE)[see] for x in (K, V))
                want[r, h], _ = attend_f64(q[r, h], k, v, DIM ** -0.5)
            r += 1
    close(o.reshape(-1, DIM), want.reshape(-1, DIM), tol, "attention")


@pytest.mark.parametrize("kind", [F16, BF16, Q8_0])
def test_prompt_then_drafts(kind):
    rng = synth.rng_for(61, kind, 0)
    W, W64 = model(rng)
    n_pages = SEQS * PAGES
    cache = g.KvCache.empty(kind, n_pages, KV_HEADS, DIM, PAGE, device=DEV)
    table = rng.permutation(n_pages).astype(np.int32).reshape(SEQS, PAGES)
    T, max_len = dev(table), PAGES * PAGE
    freqs64 = 500000.0 ** (-np.arange(DIM // 2) / (DIM // 2))
    freqs = torch.tensor(freqs64, device=DEV)
    qn, kn = (rng.uniform(0.5, 1.5, (2, DIM))).astype(np.float32)

    def turn(q, k, slot):
        q, k = q.view(len(q), HEADS, DIM), k.view(len(k), KV_HEADS, DIM)
        a, b = g.gguf_qk_rope(q, k, slot, freqs, q_norm=dev(qn), k_norm=dev(kn), eps=1e-6)
        pos = host(slot)[None]
        tol = 2e-2 if q.dtype is torch.bfloat16 else 1e-4
        close(as_f64(a), rope_f64(as_f64(q), pos, freqs64, norm=qn, eps=1e-6), tol, "q turned")
        close(as_f64(b), rope_f64(as_f64(k), pos, freqs64, norm=kn, eps=1e-6), tol, "k turned")
        return a, b

    # the prompts
    seq = np.repeat(np.arange(SEQS), PROMPTS).astype(np.int32)
    slot = np.concatenate([np.arange(p) for p in PROMPTS]).astype(np.int32)
    X = dev(f32_to_bf16_bits((0.05 * rng.standard_normal((len(seq), HIDDEN))).astype(np.float32)).view(np.int16)).view(torch.bfloat16)
    q, k, v = g.gguf_qmatmul_q4_k_multi([W["q"], W["k"], W["v"]], X)
    q, k = turn(q, k, dev(slot))
    g.gguf_kv_append(cache, k.flatten(1), v, T, dev(slot), seq=dev(seq))
    lengths = np.array(PROMPTS, np.int32)
    starts = dev(np.concatenate([[0], np.cumsum(PROMPTS)]).astype(np.int32))
    o = g.gguf_attn_extend(cache, q.flatten(1), T, dev(lengths), max_len, row_start=starts, window=WINDOW, sinks=SINKS)
    check_attention(as_f64(o), as_f64(q), cache, kind, table, lengths, PROMPTS, 3e-2)
    y = g.gguf_qmatmul_q4_k(W["o"], o)
    close(as_f64(y), as_f64(o) @ W64["o"].T, 2e-2, "output projection")

    # drafted tokens: 0 to 4 of them behind the last accepted one, as rows of one batch
    seen = set()
    for step in range(8):
        say("step", step)
        rows = [1 + int(rng.integers(0, DRAFTS + 1)) for _ in range(SEQS)]
        n = sum(rows)
        starts64 = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        seq = np.repeat(np.arange(SEQS), rows).astype(np.int32)
        slot = np.concatenate([lengths[s] + np.arange(rows[s]) for s in range(SEQS)]).astype(np.int32)
        x = (0.05 * rng.standard_normal((n, HIDDEN))).astype(np.float32)
        q, k, v = g.gguf_qmatmul_f32_q4_k_multi([W["q"], W["k"], W["v"]], dev(x))
        q, k = turn(q, k, dev(slot))
        g.gguf_kv_append(cache, k.flatten(1), v, T, dev(slot), seq=dev(seq))
        lengths = (lengths + rows).astype(np.int32)
        o = g.gguf_attn_extend(cache, q.flatten(1), T, dev(lengths), max_len, row_start=dev(starts64), window=WINDOW, sinks=SINKS)
        check_attention(host(o), as_f64(q), cache, kind, table, lengths, rows, 1e-4)
        y = g.gguf_qmatmul_f32_q4_k(W["o"], o)
        logits = g.gguf_qmatmul_f32_q4_k(W["head"], (y / y.square().mean().sqrt() * 0.05).contiguous())
        draft = logits + 0.5 * torch.randn(logits.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(step))
        p = torch.softmax(draft.double(), -1).cpu().numpy()
        tokens = np.array([rng.choice(VOCAB, p=r / r.sum()) for r in p], np.int32)
        u, un = rng.random(n).astype(np.float32), rng.random(SEQS).astype(np.float32)
        r = g.gguf_verify_draft(logits, dev(tokens), dev(u), dev(un), dev(starts64), draft=draft)
        acc, nxt, prob = verify_f64(host(logits), host(draft), tokens, u, un, starts64)
        assert np.array_equal(host(r.accepted), acc) and np.array_equal(host(r.next_tokens), nxt)
        assert np.allclose(host(r.accept_prob), prob, rtol=1e-6)
        lengths = np.minimum(lengths - rows + 1 + acc, max_len - DRAFTS - 1).astype(np.int32)   # refused drafts leave the cache
        seen |= set(acc.tolist())
    assert len(seen) > 2


def test_captured_step_replays_like_the_eager_one():
    rng = synth.rng_for(62, 0, 0)
    W, _ = model(rng)
    n_pages, rows = SEQS * PAGES, DRAFTS + 1
    T = dev(rng.permutation(n_pages).astype(np.int32).reshape(SEQS, PAGES))
    freqs = torch.tensor(500000.0 ** (-np.arange(DIM // 2) / (DIM // 2)), device=DEV)
    norm = dev(rng.uniform(0.5, 1.5, DIM).astype(np.float32))
    x = torch.zeros((SEQS * rows, HIDDEN), device=DEV)
    tokens = torch.zeros(SEQS * rows, dtype=torch.int32, device=DEV)
    u, un = torch.zeros(SEQS * rows, device=DEV), torch.zeros(SEQS, device=DEV)
    starts = dev(np.arange(0, SEQS * rows + 1, rows).astype(np.int32))
    seq = dev(np.repeat(np.arange(SEQS), rows).astype(np.int32))
    offset = dev(np.tile(np.arange(rows), SEQS).astype(np.int32))
    max_len = PAGES * PAGE

    def fresh():
        return g.KvCache.empty(F16, n_pages, KV_HEADS, DIM, PAGE, device=DEV), torch.zeros(SEQS, dtype=torch.int32, device=DEV)

    def step(cache, lengths):
        q, k, v = g.gguf_qmatmul_f32_q4_k_multi([W["q"], W["k"], W["v"]], x)
        slot = lengths[seq.long()] + offset
        q, k = g.gguf_qk_rope(q.view(-1, HEADS, DIM), k.view(-1, KV_HEADS, DIM), slot, freqs, q_norm=norm, k_norm=norm)
        g.gguf_kv_append(cache, k.flatten(1), v, T, slot, seq=seq)
        lengths += rows
        o = g.gguf_attn_extend(cache, q.flatten(1), T, lengths, max_len, row_start=starts, window=WINDOW, sinks=SINKS)
        logits = g.gguf_qmatmul_f32_q4_k(W["head"], g.gguf_qmatmul_f32_q4_k(W["o"], o))
        r = g.gguf_verify_draft(logits, tokens, u, un, starts)
        lengths += r.accepted - DRAFTS
        return o, r

    eager, graphed = fresh(), fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # warm the stream's scratch slot outside the capture
        step(*fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go, gr = step(*graphed)
    for i in range(20):
        x.copy_(dev((0.05 * rng.standard_normal(x.shape)).astype(np.float32)))
        tokens.copy_(dev(rng.integers(0, VOCAB, SEQS * rows).astype(np.int32)))
        u.copy_(dev((1e-3 * rng.random(SEQS * rows)).astype(np.float32)))
        un.copy_(dev(rng.random(SEQS).astype(np.float32)))
        eo, er = step(*eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(eo), host(go)), i
        for a, b in zip(er, gr):
            assert np.array_equal(host(a), host(b)), i
        assert np.array_equal(host(eager[1]), host(graphed[1]))
        assert np.array_equal(host(eager[0].k), host(graphed[0].k)) and np.array_equal(host(eager[0].v), host(graphed[0].v))
    g.gguf_qk_stream_release(side)
    g.gguf_qk_stream_release()
