"""The cache, attention, eviction and log probabilities where byte offsets pass 32
bits and batches are large, and calls that overlap in time."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.serving import evict_moves
from tests.serving_util import DEV, TYPES, U, attend_reference, check_bound, dev, host, make
from tests.test_gpu_kv_cache import append_reference

pytestmark = pytest.mark.gpu

OFFSET = 1 << 32


def say(*a):
    print(*a, flush=True)


def moved_up(d):
    """d's cache with its pages behind the first 4 GiB of K and of V: the cache,
    its table, and the page ids moved by."""
    page = d["k"].shape[1]
    base = OFFSET // page + 3
    k, v = (torch.empty((base + d["n_pages"], page), dtype=torch.uint8, device=DEV) for _ in range(2))
    k[base:], v[base:] = dev(d["k"]), dev(d["v"])
    w = torch.empty((base + d["n_pages"], d["hkv"], d["ps"]), dtype=torch.float32, device=DEV)
    p = torch.empty(w.shape, dtype=torch.int32, device=DEV)
    w[base:], p[base:] = dev(d["weight"]), dev(d["pos"])
    return g.KvCache(k, v, d["type"], d["hkv"], d["dim"], d["ps"], weight=w, pos=p), d["table"] + base, base


@pytest.mark.parametrize("kind", list(TYPES))
def test_pages_behind_four_gigabytes(kind):
    rng = np.random.default_rng(41)
    d = make(rng, TYPES[kind], [700, 300], 3, 4, 2, 256, 256, planes=True)
    n_pages = d["n_pages"]
    cache, table, base = moved_up(d)
    say("attend", kind)
    got = host(g.gguf_attn_decode(cache, dev(d["q"]), dev(table), dev(d["lengths"]), 700, track=True))
    want, bound, weights = attend_reference(d, 1 / 16)
    check_bound(got, want, bound, kind)
    w = host(cache.weight[base:])
    grown = w.astype(np.float64) - d["weight"]
    assert np.allclose(grown.sum(), 2 * 4, rtol=1e-4)
    d["weight"] = w
    # two tokens behind the sequences' ends
    say("append", kind)
    k, v = (rng.standard_normal((2, 512)).astype(np.float32) for _ in range(2))
    slot = np.array([700, 300], np.int32)
    kb, vb, w, p = append_reference(d, k, v, d["table"], slot, None, None)
    g.gguf_kv_append(cache, dev(k), dev(v), dev(table), dev(slot))
    assert np.array_equal(host(cache.k.view(-1, d["k"].shape[1])[base:]), kb)
    assert np.array_equal(host(cache.v.view(-1, d["k"].shape[1])[base:]), vb)
    assert np.array_equal(host(cache.pos[base:]), p)
    # down to 256 slots
    say("evict", kind)
    pos = rng.permutation(n_pages * 256).astype(np.int32).reshape(n_pages, 1, 256).repeat(2, 1)
    cache.pos[base:] = dev(pos)
    weight = host(cache.weight[base:])
    lengths = dev(np.array([701, 301], np.int32))
    g.gguf_kv_evict(cache, dev(table), lengths, 701, 256, recent=8)
    assert host(lengths).tolist() == [256, 256]
    got_w, got_k = host(cache.weight[base:]), host(cache.k.view(-1, d["k"].shape[1])[base:])
    for s, n in enumerate((701, 301)):
        at = np.arange(n)
        page, i = d["table"][s][at // 256], at % 256
        for h in range(2):
            _, sources, holes = evict_moves(weight[page, h, i], pos[page, h, i], 256, 8)
            for src, to in zip(sources, holes):
                assert got_w[page[to], h, i[to]] == weight[page[src], h, i[src]]
                if kind != "q8_0":
                    rows_new = got_k[page[to]].reshape(2, 256, -1)[h, i[to]]
                    assert np.array_equal(rows_new, kb[page[src]].reshape(2, 256, -1)[h, i[src]])


def test_rows_four_gigabytes_apart():
    """Row strides past 32 bits: logits, and the tokens of an append."""
    rng = np.random.default_rng(42)
    stride, vocab = (OFFSET // 4) + 8, 5000
    buf = torch.empty(stride + vocab, dtype=torch.float32, device=DEV)
    x = (3 * rng.standard_normal((2, vocab))).astype(np.float32)
    rows = torch.as_strided(buf, (2, vocab), (stride, 1))
    rows[0], rows[1] = dev(x[0]), dev(x[1])
    r = g.gguf_logprobs(rows, dev(np.array([[7], [4999]], np.int32)), top_k=3)
    e = x.astype(np.float64)
    lse = np.log(np.exp(e - e.max(1, keepdims=True)).sum(1)) + e.max(1)
    assert np.array_equal(host(r.top_ids), np.argsort(-e, axis=1, kind="stable")[:, :3])
    # value, logarithm and both differences rounded, sums of 5000 terms
    assert np.abs(host(r.token_logprobs)[:, 0] - (e[[0, 1], [7, 4999]] - lse)).max() <= 5200 * U
    d = make(rng, TYPES["bf16"], [3, 3], 1, 2, 1, 64, 16, planes=True, poisoned=False)
    k = (rng.standard_normal((2, 64))).astype(np.float32)
    rows = torch.as_strided(buf, (2, 64), (stride, 1))
    rows[0], rows[1] = dev(k[0]), dev(k[1])
    kb, vb, _, _ = append_reference(d, k, k, d["table"], np.array([3, 4]), None, None)
    g.gguf_kv_append(d["cache"], rows, rows, dev(d["table"]), dev(np.array([3, 4], np.int32)))
    assert np.array_equal(host(d["cache"].k), kb) and np.array_equal(host(d["cache"].v), vb)


def test_many_short_sequences():
    rng = np.random.default_rng(43)
    lengths = rng.integers(0, 20, 3000)
    d = make(rng, TYPES["f16"], lengths, 2, 2, 1, 64, 16, planes=True, poisoned=False)
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 20, track=True))
    want, bound, _ = attend_reference(d, 1 / 8)
    check_bound(got, want, bound, "many")
    grown = host(d["cache"].weight).astype(np.float64) - d["weight"]
    assert np.allclose(grown.sum(), 2 * (lengths > 0).sum(), rtol=1e-4)
    cut = dev(d["lengths"])
    g.gguf_kv_evict(d["cache"], dev(d["table"]), cut, 20, 5)
    assert np.array_equal(host(cut), np.minimum(lengths, 5))


def test_two_streams_at_once():
    """Two batches on two streams, each with its workspace, give what each gives alone."""
    rng = np.random.default_rng(44)
    ds = [make(rng, TYPES["bf16"], rng.integers(1, 4000, 16), 32, 16, 4, 128, 128, poisoned=False) for _ in range(2)]
    args = [(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 4096) for d in ds]
    alone = [host(g.gguf_attn_decode(*a)) for a in args]
    x = [dev(rng.standard_normal((8, 50000)).astype(np.float32)) for _ in ds]
    alone_top = [host(g.gguf_logprobs(v, top_k=40).top_logprobs) for v in x]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got, top = [[], []], [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append(g.gguf_attn_decode(*args[i], stream=st))
            top[i].append(g.gguf_logprobs(x[i], top_k=40, stream=st).top_logprobs)
    torch.cuda.synchronize()
    for i in range(2):
        for o, t in zip(got[i], top[i]):
            assert np.array_equal(host(o), alone[i]) and np.array_equal(host(t), alone_top[i])
