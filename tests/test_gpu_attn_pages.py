"""Attention of several new tokens where a block reads more than 64 pages (whose ids it
fetches 64 at a time), past pages that are left out, in calls of which one part decides
the kernel for another, and against the same rows in other calls; against the fp64
oracle."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
import tests.tokens_util as tokens_util
from oracle.tokens import visible_slots
from tests.serving_util import TYPES, dev, host
from tests.tokens_util import BF16, as_f64, check_rows, extend, extend_reference, make_rows

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def long_among_short(rng, kind, seqs, heads, hkv, dim, ps, long=5000):
    """One sequence of 40 rows behind a long context first, then short ones whose pages are
    the long one's in other orders. Tiles times kv heads fill the device, so that positions
    are not split: a block of the long sequence walks over all its pages."""
    d = make_rows(rng, TYPES[kind], [long], [40], -(-long // ps), heads, hkv, dim, ps, True)
    rows = np.concatenate([[40], rng.integers(33, 41, seqs - 1)])
    d["lengths"] = np.concatenate([[long], rows[1:] + rng.integers(0, 30, seqs - 1)]).astype(np.int32)
    d["table"] = np.stack([np.roll(d["table"][0], -s) for s in range(seqs)])   # the last page, part of it NaN, stays far behind
    d["rows"], d["starts"] = list(rows), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    d["Q"], d["q"] = tokens_util.as_type(2.0 * rng.standard_normal((int(rows.sum()), heads * dim)), True)
    return d


@pytest.mark.parametrize("dim,ps", [(64, 16), (64, 64), (96, 16), (128, 16), (128, 64), (192, 64), (256, 16)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_blocks_of_more_pages_than_lanes(kind, dim, ps):
    # 4 kv heads: two groups of waves where the registers hold them (up to dim 128); 16: one;
    # 70: more sequences than lanes
    for seqs, hkv in ((64, 4), (64, 16), (70, 16)) if dim <= 128 else ((64, 4), (70, 4)):
        rng = np.random.default_rng([41, dim, ps, seqs, hkv])
        d = long_among_short(rng, kind, seqs, hkv, hkv, dim, ps)
        only = {(0, 0), (0, 17), (0, 39), (1, 3), (seqs - 1, 32)}
        for window, sinks in ((0, 0), (3000, 40), (2100, 1500)):
            say("pages", kind, dim, ps, seqs, hkv, window, sinks)
            got = as_f64(extend(d, window=window, sinks=sinks))
            assert np.isfinite(got).all()
            check_rows(d, got, *extend_reference(d, dim ** -0.5, window, sinks, only=only), (window, sinks))


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_split_positions_of_more_pages_than_lanes(kind, dim):
    # a chunk of 900 rows behind a context in two to four splits of 79 to 200 pages of 16, and under a loose bound
    rng = np.random.default_rng([42, dim])
    d = make_rows(rng, TYPES[kind], [6000], [900], 375, 16, 8, dim, 16, True)
    only = {(0, j) for j in (0, 15, 16, 500, 898, 899)}
    for max_len, window, sinks in ((6000, 0, 0), (20000, 0, 0), (6000, 5300, 100)):
        need = g.gguf_attn_extend_workspace(d["cache"], torch.bfloat16, 1, 900, 16, max_len, window, sinks)
        say("split pages", kind, dim, max_len, window, need)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN
        got = as_f64(extend(d, max_len=max_len, window=window, sinks=sinks, workspace=ws))
        assert np.isfinite(got).all()
        check_rows(d, got, *extend_reference(d, dim ** -0.5, window, sinks, only=only), (max_len, window, sinks))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_pages_left_out(kind, ps, bf16, monkeypatch):
    # the first page, ones in the middle, one past the 64th, the last: of every sequence
    pages = 90 if ps < 256 else 22
    bad = [0, 5, 13, pages - 20, pages - 1]
    monkeypatch.setattr(tokens_util, "visible_slots", lambda *a: (lambda i: i[~np.isin(i // ps, bad)])(visible_slots(*a)))
    for dim, seqs, hkv in ((64, 64, 4), (128, 64, 16)) if bf16 else ((64, 3, 4),):
        rng = np.random.default_rng([43, ps, dim, bf16])
        long = (pages - 1) * ps + ps // 2 + 3
        d = long_among_short(rng, kind, seqs, hkv, hkv, dim, ps, long)
        if not bf16:
            d["bf16"], d["Q"] = False, dev(d["q"].astype(np.float32))
        # a roll apart, the same entries of every row
        table = d["table"].copy()
        table[:, bad] = np.array([-1, d["n_pages"], 2 ** 31 - 1, -(2 ** 31), -7], np.int32)
        only = {(0, 0), (0, 20), (0, 39), (1, 2), (seqs - 1, 32)}
        for window, sinks in ((0, 0), (2 * ps, 3 * ps)):
            say("bad pages", kind, ps, dim, bf16, window)
            got = as_f64(extend(dict(d, table=table), window=window, sinks=sinks))
            assert np.isfinite(got).all()
            check_rows(d, got, *extend_reference(d, dim ** -0.5, window, sinks, only=only), (dim, window))


@pytest.mark.parametrize("kind", list(TYPES))
def test_every_row_in_other_calls(kind):
    # the newest 300 of 400 tokens in one call, and the same rows in calls of 100, 37 and 163
    # (above and below the pairs where the kernel changes) and one by one
    rng = np.random.default_rng(44)
    d = make_rows(rng, TYPES[kind], [400], [300], 7, 4, 2, 128, 64, True)
    whole = as_f64(extend(d)).reshape(300, 4, 128)
    want, bound = extend_reference(d, 128 ** -0.5)
    assert (np.abs(whole - want) <= bound).all()
    for cuts in ((0, 100, 137, 300), (0, 3, 10, 300), (292, 293, 294, 295, 296, 297, 298, 299, 300)):
        for a, b in zip(cuts, cuts[1:]):
            part = dict(d, lengths=np.array([100 + b], np.int32), starts=np.array([0, b - a], np.int32), Q=d["Q"][a:b])
            got = as_f64(extend(part)).reshape(b - a, 4, 128)
            assert (np.abs(got - whole[a:b]) <= 2 * bound[a:b]).all(), (a, b)


@pytest.mark.parametrize("kind", list(TYPES))
def test_bf16_single_tokens_beside_the_decode_call(kind):
    rng = np.random.default_rng(45)
    lengths = [1, 0, 700, 33, 2000]
    d = make_rows(rng, TYPES[kind], lengths, [1] * 5, 32, 8, 2, 128, 64, True)
    got = as_f64(extend(d, starts=False)).reshape(5, 8, 128)
    one = host(g.gguf_attn_decode(d["cache"], d["Q"].float(), dev(d["table"]), dev(d["lengths"]), 2000)).reshape(5, 8, 128)
    want, bound = extend_reference(d, 128 ** -0.5)
    single = extend_reference(dict(d, bf16=False), 128 ** -0.5)[1]   # of the decode call
    assert (np.abs(got - one) <= bound + single).all(), float((np.abs(got - one) - bound - single).max())
    assert not got[1].any() and not one[1].any()


@pytest.mark.parametrize("kind", list(TYPES))
def test_single_tokens_among_a_prompt(kind):
    # by the average the kernel for many rows takes all: single tokens of long contexts fill one
    # row of its tiles; fewer tiles than blocks (split) and more
    for singles, prompt, hkv in ((7, 300, 2), (31, 1200, 8), (70, 1300, 8)):
        rng = np.random.default_rng([46, singles])
        d = make_rows(rng, TYPES[kind], [3000], [1], 188, 2 * hkv, hkv, 64, 16, True)
        s = singles + 1
        d["lengths"] = rng.integers(1, 3000, s).astype(np.int32)
        d["lengths"][[0, 2]] = 3000, 0
        d["table"] = np.stack([np.roll(d["table"][0], -i) for i in range(s)])
        rows = np.ones(s, np.int64)
        # (rolled, the long one's last page with its NaNs lies 2 pages behind the others' ends or more)
        d["lengths"] = np.minimum(d["lengths"], (187 - np.arange(s)) * 16).astype(np.int32)
        d["lengths"][0] = 3000
        at = s // 2
        rows[at], d["lengths"][at] = prompt, prompt + 40
        d["rows"], d["starts"] = list(rows), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        d["Q"], d["q"] = tokens_util.as_type(2.0 * rng.standard_normal((int(rows.sum()), 2 * hkv * 64)), True)
        assert 2 * rows.sum() > 32 * s
        only = {(i, 0) for i in (0, 1, 2, 3, s - 1)} | {(at, j) for j in (0, 31, 100, prompt - 1)}
        for window, sinks in ((0, 0), (1000, 4)):
            say("mixed", kind, singles, prompt, hkv, window)
            got = as_f64(extend(d, window=window, sinks=sinks))
            assert np.isfinite(got).all() and not got[2].any()
            check_rows(d, got, *extend_reference(d, 0.125, window, sinks, only=only), (singles, window))


@pytest.mark.parametrize("bf16", [False, True])
def test_split_calls_with_starts_outside(bf16):
    # of entries outside the rows the part within counts; rows of no sequence stay, whatever the
    # workspace holds
    rng = np.random.default_rng([47, bf16])
    d = make_rows(rng, BF16, [2900, 1800, 700], [25, 40, 13], 182, 4, 2, 64, 16, bf16, extra=9)
    n = 87
    need = g.gguf_attn_extend_workspace(d["cache"], d["Q"].dtype, 3, n, 4, 2900)
    assert need > 0
    for starts in ([4, 29, 69, 82], [-5, 24, 64, 500], [0, 0, 30, 30], [80, 90, 100, 2 ** 31 - 1], [-(2 ** 31), -1, 0, 3],
                   [-9, 87, 87, 87], [87, 87, 90, 95], [70, 30, 30, 76]):
        inside = np.clip(np.array(starts, np.int64), 0, n)
        rows = [max(0, int(b - a)) for a, b in zip(inside, inside[1:])]
        out = torch.full_like(d["Q"], 7.0)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        e = dict(d, starts=np.array(starts, np.int32), rows=rows)
        say("starts", starts, bf16)
        got = as_f64(extend(e, out=out, workspace=ws))
        mine = np.zeros(n, bool)
        for a, m in zip(inside, rows):
            mine[a:a + m] = True
        assert (got[~mine] == 7).all() and np.isfinite(got[mine]).all(), starts
        want, bound = extend_reference(dict(e, starts=inside), 0.125)
        check_rows(e, got, want, bound, starts)
