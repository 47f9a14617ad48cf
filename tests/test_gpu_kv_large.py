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


@pytest.mark.parametrize("kind", list(TYPES))
def test_bounds_far_above_the_lengths(kind):
    """Chunks are cut to the lengths on the device: any bound, any mix of lengths,
    with a window, tracked, under a bound that cuts, and replayed with new lengths."""
    rng = np.random.default_rng(45)
    for lengths in ([3000, 1, 0, 2047], [5000], [700] * 9, list(rng.integers(0, 1500, 64))):
        d = make(rng, TYPES[kind], lengths, -(-max(lengths) // 64), 4, 2, 64, 64, planes=True)
        for max_len in (max(lengths), 40000, 300000, 1200):
            for window in (0, 1111):
                say(kind, len(lengths), max_len, window)
                before = host(d["cache"].weight).astype(np.float64)
                got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), max_len,
                                              window=window, track=True))
                want, bound, _ = attend_reference(d, 1 / 8, window=window, cut=max_len)
                check_bound(got, want, bound, (kind, max_len, window))
                grown = host(d["cache"].weight).astype(np.float64) - before
                assert np.allclose(grown.sum(), 4 * (np.asarray(lengths) > 0).sum(), rtol=1e-3)


def test_captured_under_a_far_bound():
    rng = np.random.default_rng(46)
    d = make(rng, TYPES["q8_0"], [6000, 6000, 6000], 47, 8, 2, 128, 128, planes=True, poisoned=False)
    q, t, n = dev(d["q"]), dev(d["table"]), dev(d["lengths"])
    out = torch.empty_like(q)
    ws = torch.empty(g.gguf_attn_decode_workspace(d["cache"], 3, 8, 200000, True), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g.gguf_attn_decode(d["cache"], q, t, n, 200000, track=True, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gguf_attn_decode(d["cache"], q, t, n, 200000, track=True, out=out, workspace=ws)
    for lengths in ([10, 6000, 0], [300, 301, 302], [5999, 1, 4096], [6000, 6000, 6000]):
        d["lengths"] = np.array(lengths, np.int32)
        n.copy_(dev(d["lengths"]))
        graph.replay()
        got = host(out)
        assert np.array_equal(got, host(g.gguf_attn_decode(d["cache"], q, t, n, 200000)))
        want, bound, _ = attend_reference(d, 128 ** -0.5)
        check_bound(got, want, bound, lengths)


def scaled(d, factor):
    """Multiplies V's Q8_0 scales by factor [head, block, slot of the sequence] (one
    sequence), rounded to fp16, in the arrays and on the device."""
    nb, ps = d["dim"] // 32, d["ps"]
    v = d["v"].reshape(d["n_pages"], d["hkv"], -1)
    scales = v[..., ps * d["dim"]:].copy().view(np.float16).reshape(d["n_pages"], d["hkv"], nb, ps)
    n = factor.shape[-1]
    at = np.arange(n)
    page, slot = d["table"][0][at // ps], at % ps
    for h in range(d["hkv"]):
        for b in range(nb):
            scales[page, h, b, slot] = (scales[page, h, b, slot].astype(np.float64) * factor[h, b]).astype(np.float16)
    v[..., ps * d["dim"]:] = scales.reshape(d["n_pages"], d["hkv"], -1).view(np.uint8)
    d["cache"].v.copy_(dev(d["v"]).view(d["cache"].v.shape))


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_q8_0_scales_of_all_magnitudes(dim):
    """V's scales enter fp16 times powers of two that follow the greatest met: blocks
    of unlike size, scales that grow or fall along the sequence, the type's greatest,
    subnormal and zero ones. Values below the greatest by 2^-19 keep the full bound."""
    rng = np.random.default_rng(dim)
    n, nb = 900, dim // 32
    ramp = np.linspace(0, 1, n)
    cases = {
        "blocks": np.exp2(rng.integers(-12, 21, (2, nb, 1)).astype(float)) * np.ones(n),
        "rising": np.exp2(18 * ramp - 9) * np.ones((2, nb, 1)),
        "falling": np.exp2(9 - 18 * ramp) * np.ones((2, nb, 1)),
        "greatest": np.full((2, nb, n), 65504 / 0.03),
        "subnormal": np.full((2, nb, n), 2.0 ** -17),
        "zeros": np.where(rng.random((2, nb, n)) < 0.5, 0.0, 1.0),
        "negative": np.where(rng.random((2, nb, n)) < 0.5, -1.0, 4.0),
    }
    for name, factor in cases.items():
        d = make(rng, TYPES["q8_0"], [n], 15, 6, 2, dim, 64, poisoned=False)
        scaled(d, factor)
        say(dim, name)
        got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), n))
        want, bound, _ = attend_reference(d, dim ** -0.5)
        check_bound(got, want, bound, (dim, name))
    d = make(rng, TYPES["q8_0"], [n], 15, 6, 2, dim, 64, poisoned=False)
    scaled(d, np.zeros((2, nb, n)))
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), n))
    assert not got.any()


@pytest.mark.parametrize("ps", [16, 32, 256])
@pytest.mark.parametrize("kind,heads,hkv", [("f16", 34, 1), ("bf16", 5, 5), ("q8_0", 20, 1), ("q8_0", 8, 4)])
def test_far_bounds_of_page_sizes_and_head_layouts(kind, heads, hkv, ps):
    rng = np.random.default_rng([47, ps, heads])
    lengths = [2500, 1029, 33, 0, 511]
    d = make(rng, TYPES[kind], lengths, -(-2500 // ps) + 1, heads, hkv, 96, ps)
    for max_len in (2500, 70000, 1 << 25):
        for window in (0, 300):
            say(kind, heads, hkv, ps, max_len, window)
            got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), max_len,
                                          window=window))
            want, bound, _ = attend_reference(d, 96 ** -0.5, window=window)
            check_bound(got, want, bound, (kind, ps, max_len, window))


def test_bound_of_zero():
    rng = np.random.default_rng(48)
    d = make(rng, TYPES["f16"], [30, 20], 1, 4, 2, 64, 32, planes=True)
    out = torch.full((2, 4, 64), 7.0, device=DEV)
    g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 0, track=True, out=out)
    assert not host(out).any()
    assert np.array_equal(host(d["cache"].weight), d["weight"])
    k, v = host(d["cache"].k), host(d["cache"].v)
    n = dev(d["lengths"])
    g.gguf_kv_evict(d["cache"], dev(d["table"]), n, 0, 25)   # slots behind the bound are not looked at
    assert host(n).tolist() == [25, 20]
    assert np.array_equal(host(d["cache"].k), k) and np.array_equal(host(d["cache"].v), v)
