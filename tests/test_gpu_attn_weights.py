"""The attention weights that a tracked call adds, slot by slot, wherever the split
over positions, the window, the head layout or the cache's offsets could put
them in the wrong place; and scales below zero."""

import numpy as np
import pytest

import gguf_block_quant_dequant_amd as g
from oracle.serving import attend_f64, sequence_f64
from tests.serving_util import TYPES, U, check_bound, dev, host, make, values
from tests.test_gpu_kv_large import moved_up

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def reference(d, scale, window=0, cut=None):
    """(out, its bound, growth of the weights, its bound), the first two by sequence and
    head, the others by page, head and slot.

    A score is off by es = (4 U + 2^-22 + 3 dim U) |scale| max sum|q k| (the parts of
    q, the products' sums, scale and unit); the exponential by 4 U of its argument
    beside it, 4 U of its value and 2^-22 (the weights' parts). The normalized
    weight carries this twice (its own and the sum's) and 8 n + 128 roundings of
    sums and rescales; the output sums weights times |v|, the growth the heads of
    a group, added to the slot's weight once."""
    K, V = values(d)
    group, ps = d["heads"] // d["hkv"], d["ps"]
    out = np.zeros((len(d["lengths"]), d["heads"], d["dim"]))
    bound = np.full(out.shape, 1e-30)
    grown = np.zeros((d["n_pages"], d["hkv"], ps))
    grown_bound = np.zeros(grown.shape)
    for s, n in enumerate(d["lengths"]):
        n = max(0, int(n) if cut is None else min(int(n), cut))
        if n == 0:
            continue
        first = max(0, n - window) if window else 0
        at = np.arange(first, n)
        page, slot = d["table"][s][at // ps], at % ps
        for j in range(d["heads"]):
            h = j // group
            k, v = (sequence_f64(x, d["table"][s], h, n, ps)[first:] for x in (K, V))
            q = d["q"][s, j].astype(np.float64)
            out[s, j], p = attend_f64(q, k, v, scale)
            mag = abs(scale) * (np.abs(k) @ np.abs(q)).max()
            ew = (8 * U + 2.0 ** -22 + 3 * d["dim"] * U) * mag + 4 * U + 2.0 ** -22
            rel = 2 * ew + (8 * len(p) + 128) * U
            bound[s, j] += rel * (p @ np.abs(v))
            grown[page, h, slot] += p
            grown_bound[page, h, slot] += rel * p
    return out, bound, grown, grown_bound


def check_weights(d, before, after, grown, bound, what):
    """after: the plane on the device, as numbers of `before` plus the growth."""
    group = d["heads"] // d["hkv"]
    assert np.array_equal(after[grown == 0].view(np.uint32), before[grown == 0].view(np.uint32)), what
    off = np.abs(after.astype(np.float64) - (before.astype(np.float64) + grown))
    over = off - (bound + (group + 2) * U * (np.abs(before) + grown) + 1e-36)
    assert (over <= 0).all(), (what, float(over.max()), np.argwhere(over > 0)[:4])


@pytest.mark.parametrize("heads,hkv", [(1, 1), (5, 1), (16, 4), (17, 1), (40, 1), (66, 2), (14, 2)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_head_layouts(kind, heads, hkv):
    rng = np.random.default_rng([heads, hkv, 100])
    d = make(rng, TYPES[kind], [5, 200, 333, 0, 1100], 9, heads, hkv, 128, 128, planes=True)
    for window in (0, 77):
        before = host(d["cache"].weight)
        got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 1100, track=True,
                                      window=window))
        want, bound, grown, gb = reference(d, 128 ** -0.5, window)
        check_bound(got, want, bound, (kind, heads, hkv, window))
        check_weights(d, before, host(d["cache"].weight), grown, gb, (kind, heads, hkv, window))


@pytest.mark.parametrize("kind", list(TYPES))
def test_far_bounds_windows_and_cuts(kind):
    rng = np.random.default_rng(101)
    for lengths in ([3000, 1, 0, 2047], [5000], [700] * 9, list(rng.integers(0, 1500, 64)),
                    list(rng.integers(0, 400, 70))):
        d = make(rng, TYPES[kind], lengths, -(-max(lengths) // 64), 4, 2, 64, 64, planes=True)
        for max_len in (max(lengths), 40000, 1200):
            for window in (0, 33, 1111):
                say(kind, len(lengths), max_len, window)
                before = host(d["cache"].weight)
                got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), max_len,
                                              window=window, track=True))
                want, bound, grown, gb = reference(d, 1 / 8, window, cut=max_len)
                check_bound(got, want, bound, (kind, max_len, window))
                check_weights(d, before, host(d["cache"].weight), grown, gb, (kind, max_len, window))


@pytest.mark.parametrize("ps", [16, 32, 256])
@pytest.mark.parametrize("dim", [96, 192, 256])
def test_page_sizes_and_head_dims(dim, ps):
    for kind in TYPES:
        rng = np.random.default_rng([dim, ps, 102])
        d = make(rng, TYPES[kind], [2500, 1029, 33, 0, 511], -(-2500 // ps) + 1, 6, 2, dim, ps, planes=True)
        for window in (0, 300):
            say(kind, dim, ps, window)
            before = host(d["cache"].weight)
            got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 2500,
                                          window=window, track=True))
            want, bound, grown, gb = reference(d, dim ** -0.5, window)
            check_bound(got, want, bound, (kind, dim, ps, window))
            check_weights(d, before, host(d["cache"].weight), grown, gb, (kind, dim, ps, window))


@pytest.mark.parametrize("kind", list(TYPES))
def test_pages_behind_four_gigabytes(kind):
    rng = np.random.default_rng(103)
    d = make(rng, TYPES[kind], [700, 300], 3, 4, 2, 256, 256, planes=True)
    cache, table, base = moved_up(d)
    say("attend", kind)
    g.gguf_attn_decode(cache, dev(d["q"]), dev(table), dev(d["lengths"]), 700, track=True)
    _, _, grown, gb = reference(d, 1 / 16)
    check_weights(d, d["weight"], host(cache.weight[base:]), grown, gb, kind)


@pytest.mark.parametrize("scale", [-0.02, -0.125, -0.3])
@pytest.mark.parametrize("kind", list(TYPES))
def test_scales_below_zero(kind, scale):
    rng = np.random.default_rng(104)
    d = make(rng, TYPES[kind], [700, 31, 300], 11, 4, 1, 64, 64, planes=True)
    got = host(g.gguf_attn_decode(d["cache"], dev(d["q"]), dev(d["table"]), dev(d["lengths"]), 700, scale=scale,
                                  track=True))
    want, bound, grown, gb = reference(d, scale)
    # the bound tells the outputs from those of the opposite scale, and from zeros
    other = reference(d, -scale)[0]
    assert np.median(bound / np.abs(want)) < 0.05 and (np.abs(other - want) > 2 * bound).mean() > 0.9
    check_bound(got, want, bound, (kind, scale))
    check_weights(d, d["weight"], host(d["cache"].weight), grown, gb, (kind, scale))
