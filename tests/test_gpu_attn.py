"""Attention of one new token over the paged cache, against the fp64 oracle:
every cache type and head dim, group sizes, page sizes, lengths from none to
long, windows, garbage behind the lengths, bad pages, strides, streams, graphs."""

import math

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from tests.serving_util import DEV, TYPES, U, attend_reference, check_bound, dev, host, make

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def attend(d, max_len=None, **kw):
    n = int(max(d["lengths"].max(), 1)) if max_len is None else max_len
    return g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), n, **kw)


@pytest.mark.parametrize("track", [False, True])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_types_and_head_dims(kind, dim, track):
    # lengths around the 32-position tiles, the page size and several splits
    rng = np.random.default_rng([dim, len(kind)])
    lengths = [0, 1, 2, 31, 32, 33, 63, 64, 65, 129, 300, 577]
    d = make(rng, TYPES[kind], lengths, 10, 6, 2, dim, 64, planes=True)
    say("attend", kind, dim, track)
    got = host(attend(d, track=track))
    want, bound, weights = attend_reference(d, 1 / math.sqrt(dim))
    check_bound(got, want, bound, (kind, dim))
    assert not got[0].any()   # an idle slot is zero
    w = host(d["cache"].weight)
    if not track:
        assert np.array_equal(w, d["weight"])
        return
    expect = d["weight"].astype(np.float64)
    for s, n in enumerate(lengths):
        at = np.arange(n)
        for h in range(2):
            expect[d["table"][s][at // 64], h, at % 64] += weights[s][h]
    # weights: relative error of the exponential as in the reference's bound,
    # 3 heads' sum and the addition to a value below 4
    assert np.abs(w - expect).max() <= 3 * (2e-4 + 8 * 577 * U) and np.allclose(w, expect, rtol=0, atol=3e-5)


@pytest.mark.parametrize("heads,hkv", [(1, 1), (5, 1), (8, 8), (16, 4), (16, 1), (17, 1), (40, 1), (66, 2), (14, 2)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_head_layouts(kind, heads, hkv):
    rng = np.random.default_rng([heads, hkv, 3])
    d = make(rng, TYPES[kind], [5, 200, 333], 3, heads, hkv, 128, 128, planes=True)
    got = host(attend(d, track=True))
    want, bound, weights = attend_reference(d, 1 / math.sqrt(128))
    check_bound(got, want, bound, (kind, heads, hkv))
    w = host(d["cache"].weight).astype(np.float64) - d["weight"]
    # every query head's weights sum to one
    assert np.allclose(w.sum(), 3 * heads, rtol=1e-4)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_page_sizes_and_windows(kind, ps):
    rng = np.random.default_rng([ps, 4])
    lengths = [1, 15, 16, 17, 47, 500, 1030]
    d = make(rng, TYPES[kind], lengths, -(-1030 // ps) + 1, 4, 1, 64, ps)
    for window in (0, 1, 7, 32, 33, 100, 512, 1029, 5000):
        got = host(attend(d, window=window))
        want, bound, _ = attend_reference(d, 1 / 8, window=window)
        check_bound(got, want, bound, (kind, ps, window))


@pytest.mark.parametrize("kind", list(TYPES))
def test_long_cache_and_bounds_on_the_length(kind):
    rng = np.random.default_rng(11)
    d = make(rng, TYPES[kind], [9000, 4097], 71, 8, 2, 128, 128, poisoned=False)
    for max_len in (9000, 20000, 9088, 5000, 1):   # a wider bound, one that cuts
        got = host(attend(d, max_len=max_len))
        want, bound, _ = attend_reference(d, 1 / math.sqrt(128), cut=max_len)
        check_bound(got, want, bound, (kind, max_len))
    # relative 2-norm: rounding errors that do not line up
    assert np.linalg.norm(host(attend(d)) - attend_reference(d, 1 / math.sqrt(128))[0]) <= 2e-6 * np.linalg.norm(
        attend_reference(d, 1 / math.sqrt(128))[0])


def test_lengths_past_the_table_and_negative_ones():
    rng = np.random.default_rng(12)
    d = make(rng, TYPES["bf16"], [64, 64, 64], 2, 4, 1, 64, 32, poisoned=False)
    d["lengths"] = np.array([1000, -5, 2 ** 31 - 1], np.int32)
    got = host(attend(d, max_len=4096))
    want, bound, _ = attend_reference(d, 1 / 8, cut=64)
    check_bound(got, want, bound, "cut at the table")
    assert not got[1].any()


@pytest.mark.parametrize("kind", list(TYPES))
def test_bad_pages_are_left_out(kind):
    """Ids outside the cache: their positions do not take part (their bounds are
    tested on the CPU, tests/test_kv_layout_cpu.py)."""
    rng = np.random.default_rng(13)
    d = make(rng, TYPES[kind], [130, 90, 64], 5, 4, 2, 64, 32, poisoned=False, planes=True)
    table = d["table"].copy()
    table[0, 1], table[1, 0], table[1, 2], table[2, :] = -1, d["n_pages"], 2 ** 31 - 1, -7
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(table), dev(d["lengths"]), 130, track=True))
    # the reference: the same sequences without these pages
    short = dict(d, table=d["table"].copy(), lengths=np.array([98, 32, 0], np.int32))
    short["table"][0] = d["table"][0][[0, 2, 3, 4, 1]]
    short["table"][1] = d["table"][1][[1, 0, 2, 3, 4]]
    want, bound, _ = attend_reference(short, 1 / 8)
    check_bound(got, want, bound, kind)
    assert not got[2].any()
    w = host(d["cache"].weight).astype(np.float64) - d["weight"]
    assert np.allclose(w.sum(), 8, rtol=1e-4)   # two live sequences of four heads


def test_peaked_and_flat_scores():
    # one position far above the rest; scores all equal; scores far below zero
    rng = np.random.default_rng(14)
    for kind in TYPES:
        for scale in (0.0, 3.0, -3.0):
            d = make(rng, TYPES[kind], [700], 11, 4, 1, 128, 64)
            got = host(attend(d, scale=scale))
            K = attend_reference(d, scale)
            # a scale of either sign: the magnitude bounds the scores' error
            bound = attend_reference(d, abs(scale))[1] if scale < 0 else K[1]
            p_abs = np.abs(values_max(d))
            check_bound(got, K[0], bound + (2 * ew(d, abs(scale)) * p_abs if scale < 0 else 0), (kind, scale))


def values_max(d):
    from tests.serving_util import values
    return np.nanmax(np.abs(np.where(np.isfinite(values(d)[1]), values(d)[1], 0)))


def ew(d, scale):
    from tests.serving_util import values
    k = values(d)[0]
    m = scale * np.abs(d["q"]).sum(-1).max() * np.nanmax(np.abs(np.where(np.isfinite(k), k, 0)))
    return (8 * U + 2.0 ** -22 + 3 * d["dim"] * U) * m


@pytest.mark.parametrize("factor", [2.0 ** -120, 1e-8, 1.0, 1e5, 3e30])
def test_query_magnitudes(factor):
    # the fp16 cache scales q's row by a power of two: any magnitude of q counts
    # with its full precision (the scale is undone by `scale`)
    rng = np.random.default_rng(15)
    for kind in TYPES:
        d = make(rng, TYPES[kind], [100], 2, 4, 1, 64, 64)
        base = d["q"]
        d["q"] = (base * np.float32(factor)).astype(np.float32)
        scale = float(np.float32(0.125 / factor))
        got = host(attend(d, scale=scale))
        want, bound, _ = attend_reference(d, scale)
        check_bound(got, want, bound, (kind, factor))


def test_small_and_large_cache_values():
    # subnormal fp16 keys and values, and values near fp16's top
    rng = np.random.default_rng(16)
    for kind in ("f16", "bf16"):
        for scale in (3e-7, 1e-4, 3000.0):
            d = make(rng, TYPES[kind], [257], 5, 4, 1, 64, 64, scale=scale)
            sc = float(np.float32(0.125 / scale))
            got = host(attend(d, scale=sc))
            want, bound, _ = attend_reference(d, sc)
            check_bound(got, want, bound, (kind, scale))


def test_strided_rows_and_given_outputs():
    rng = np.random.default_rng(17)
    d = make(rng, TYPES["f16"], [100, 40], 2, 4, 2, 64, 64)
    want, bound, _ = attend_reference(d, 0.125)
    wide = torch.full((2, 3 * 256), float("nan"), device=DEV)   # q between k and v of one buffer
    wide[:, 256:512] = dev(d["q"]).view(2, 256)
    out = torch.full((2, 512), 7.0, device=DEV)
    r = g.gguf_attn_decode(d["cache"], wide[:, 256:512], dev(d["table"]), dev(d["lengths"]), 128, out=out[:, :256])
    got = host(out)
    assert r.data_ptr() == out.data_ptr()
    check_bound(got[:, :256].reshape(2, 4, 64), want, bound, "strided")
    assert (got[:, 256:] == 7.0).all()
    with pytest.raises(ValueError):
        g.gguf_attn_decode(d["cache"], wide[:, 256:512].t(), dev(d["table"]), dev(d["lengths"]), 128)
    with pytest.raises(g.GgufQkArgumentError):
        g.gguf_attn_decode(d["cache"], wide[:, 1:257], dev(d["table"]), dev(d["lengths"]), 128)   # 4-byte aligned
    with pytest.raises(ValueError):
        g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"])[:1], dev(d["lengths"]), 128)
    with pytest.raises(g.GgufQkArgumentError):
        g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 128, track=True)   # no weight
    with pytest.raises(ValueError):
        g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]).long(), 128)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    with pytest.raises(g.GgufQkArgumentError):
        g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 100000, workspace=small)


def test_shared_pages_and_no_sequences():
    rng = np.random.default_rng(18)
    d = make(rng, TYPES["bf16"], [96, 96], 2, 4, 1, 64, 64, poisoned=False)
    table = d["table"].copy()
    table[1, 0] = table[0, 0]   # a common prefix page
    d["table"] = table
    got = host(attend(d))
    want, bound, _ = attend_reference(d, 0.125)
    check_bound(got, want, bound, "shared prefix")
    none = g.gguf_attn_decode(d["cache"], torch.empty((0, 4, 64), device=DEV), dev(table[:0]),
                              torch.empty(0, dtype=torch.int32, device=DEV), 64)
    assert none.shape == (0, 4, 64)


def test_identical_results_in_a_batch_alone_and_again():
    # the same bits whatever the run, and two streams at once with a workspace each
    rng = np.random.default_rng(19)
    d = make(rng, TYPES["bf16"], [3000, 17, 0, 2999], 47, 16, 4, 128, 64, poisoned=False)
    q, t, n = dev(d["q"]), dev(d["table"]), dev(d["lengths"])
    torch.cuda.synchronize()
    first = host(g.gguf_attn_decode(d["cache"], q, t, n, 3008))
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for s in streams:
            outs.append(g.gguf_attn_decode(d["cache"], q, t, n, 3008, stream=s))
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(host(o), first)


@pytest.mark.parametrize("track", [False, True])
def test_graph_replays_follow_the_lengths(track):
    """One captured call, replayed as the sequences grow: eager work and
    synchronizations between the replays; each replay is checked."""
    rng = np.random.default_rng(20)
    d = make(rng, TYPES["f16"], [600, 600], 10, 8, 2, 64, 64, poisoned=False, planes=True)
    c = d["cache"]
    q, t, n = dev(d["q"]), dev(d["table"]), dev(np.array([1, 1], np.int32))
    out = torch.empty((2, 8, 64), device=DEV)
    ws = torch.empty(max(16, g.gguf_attn_decode_workspace(c, 2, 8, 640, track)), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g.gguf_attn_decode(c, q, t, n, 640, out=out, workspace=ws, track=track)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gguf_attn_decode(c, q, t, n, 640, out=out, workspace=ws, track=track)
    for lengths in ([5, 600], [33, 0], [600, 599], [257, 256], [64, 1]):
        n.copy_(dev(np.array(lengths, np.int32)))
        d["lengths"] = np.array(lengths, np.int32)
        want, bound, _ = attend_reference(d, 0.125)
        out.fill_(float("nan"))
        before = host(c.weight)
        graph.replay()
        check_bound(host(out), want, bound, lengths)
        grown = host(c.weight).astype(np.float64).sum() - before.astype(np.float64).sum()
        assert np.isclose(grown, 8 * sum(x > 0 for x in lengths) if track else 0.0, rtol=1e-4, atol=1e-3)
        eager = g.gguf_attn_decode(c, q, t, n, 640)
        assert np.array_equal(host(eager), host(out))
