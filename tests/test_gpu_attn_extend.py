"""Attention of several new tokens per sequence over the paged cache, against the fp64
oracle: cache and query types, head dims, group and page sizes, ragged rows, windows
with first slots, garbage behind the lengths, bad pages, odd row_start, strides,
streams, graphs."""

import math

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.serving import attend_f64, sequence_f64
from oracle.tokens import visible_slots
from tests.serving_util import DEV, TYPES, dev, host, values
from tests.tokens_util import BF16, as_f64, check_rows, extend, extend_reference, make_rows

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def run(d, scale=None, **kw):
    sc = d["dim"] ** -0.5 if scale is None else scale
    got = as_f64(extend(d, scale=scale, **kw))
    want, bound = extend_reference(d, sc, kw.get("window", 0), kw.get("sinks", 0))
    check_rows(d, got, want, bound, {k: v for k, v in kw.items() if isinstance(v, int)})
    return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_types_and_head_dims(kind, dim, bf16):
    rng = np.random.default_rng([dim, len(kind), bf16])
    lengths = [0, 1, 2, 33, 64, 70, 129, 300, 577, 40]
    rows = [1, 1, 2, 33, 3, 5, 1, 9, 40, 0]
    d = make_rows(rng, TYPES[kind], lengths, rows, 10, 6, 2, dim, 64, bf16)
    say("extend", kind, dim, bf16)
    got = run(d)
    assert not got[0].any()   # an idle sequence's row is zero
    run(d, window=20, sinks=3)


@pytest.mark.parametrize("heads,hkv", [(1, 1), (5, 1), (8, 8), (16, 4), (16, 1), (17, 1), (40, 1), (14, 2)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_head_layouts(kind, heads, hkv):
    for bf16 in (False, True):
        rng = np.random.default_rng([heads, hkv, 3, bf16])
        d = make_rows(rng, TYPES[kind], [5, 200, 333], [2, 7, 60], 3, heads, hkv, 64, 128, bf16)
        say("heads", kind, heads, hkv, bf16)
        run(d)
        run(d, window=40, sinks=5)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_page_sizes_windows_and_first_slots(kind, bf16, ps):
    rng = np.random.default_rng([ps, 4, bf16])
    lengths, rows = [1, 17, 47, 500, 1030], [1, 4, 47, 21, 35]
    d = make_rows(rng, TYPES[kind], lengths, rows, -(-1030 // ps) + 1, 2, 1, 64, ps, bf16)
    for window, sinks in ((0, 0), (1, 0), (1, 1), (7, 4), (32, 33), (100, 16), (512, 300), (1029, 5), (5000, 1), (64, 2000)):
        say("window", window, sinks)
        run(d, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("bf16", [False, True])
def test_single_tokens_equal_the_decode_call_in_value(kind, bf16):
    rng = np.random.default_rng([5, bf16])
    lengths = [1, 0, 700, 33, 2000]
    d = make_rows(rng, TYPES[kind], lengths, [1] * 5, 32, 8, 2, 128, 64, bf16)
    run(d, starts=False)
    run(d, starts=False, window=100)
    run(d, starts=False, window=100, sinks=4)
    got = as_f64(extend(d, starts=False))
    q = d["Q"].float()
    one = host(g.gguf_attn_decode(d["cache"], q, dev(d["table"]), dev(d["lengths"]), 2000))
    if not bf16:
        assert np.allclose(got, one, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("kind", list(TYPES))
def test_long_prompt_rows(kind):
    # rows of a prompt longer than many tiles, a chunk behind 3000 slots, and a short one
    rng = np.random.default_rng([7, len(kind)])
    lengths, rows = [1500, 3700, 90], [1500, 700, 90]
    d = make_rows(rng, TYPES[kind], lengths, rows, 60, 4, 2, 128, 64, True)
    only = {(s, j) for s, m in enumerate(rows) for j in list(range(0, m, 173)) + [1, 31, 32, 63, 64, m - 2, m - 1]}
    for window, sinks in ((0, 0), (300, 4), (1000, 100)):
        got = as_f64(extend(d, window=window, sinks=sinks))
        assert np.isfinite(got).all()
        want, bound = extend_reference(d, 128 ** -0.5, window, sinks, only=only)
        check_rows(d, got, want, bound, (kind, window, sinks))


@pytest.mark.parametrize("bf16", [False, True])
def test_many_sequences_and_empty_ones(bf16):
    # more sequences than lanes, most with few rows, some with none
    rng = np.random.default_rng([8, bf16])
    lengths = rng.integers(0, 90, 150)
    rows = np.minimum(lengths, rng.integers(0, 4, 150))
    rows[70] = lengths[70] = 80
    d = make_rows(rng, BF16, lengths, rows, 6, 3, 1, 64, 16, bf16)
    run(d)
    run(d, window=9, sinks=2)


@pytest.mark.parametrize("bf16", [False, True])
def test_more_rows_than_held(bf16):
    # rows whose slot would lie before the first see nothing; bounds cut the lengths
    rng = np.random.default_rng([9, bf16])
    d = make_rows(rng, BF16, [3, 0, 40, 100], [5, 4, 60, 100], 3, 4, 2, 64, 64, bf16)
    got = run(d)
    assert not got[:2].any() and got[2].any() and not got[5:9].any() and not got[9:29].any()
    got = as_f64(extend(d, max_len=50))
    want, bound = extend_reference(d, 1 / 8, cut=50)
    check_rows(d, got, want, bound, "cut")
    assert not as_f64(extend(d, max_len=0)).any()


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_of_no_sequence_are_left(bf16):
    rng = np.random.default_rng([10, bf16])
    d = make_rows(rng, BF16, [50, 80, 60], [20, 40, 7], 2, 4, 2, 64, 64, bf16, extra=9)
    d["starts"] = np.array([4, 24, 64, 71], np.int32)   # rows 0 .. 3 and 71 on are nobody's
    out = torch.full_like(d["Q"], 7.0)
    extend(d, out=out)
    got = as_f64(out)
    assert (got[:4] == 7).all() and (got[71:] == 7).all()
    want, bound = extend_reference(d, 1 / 8)
    check_rows(d, got, want, bound, "shifted")
    # entries outside, and descending ones
    for starts in ([-5, 24, 64, 500], [70, 30, 30, 76], [0, 0, 0, 0], [80, 90, 100, 2 ** 31 - 1], [-(2 ** 31), -1, 0, 3]):
        d["starts"] = np.array(starts, np.int32)
        out = torch.full_like(d["Q"], 7.0)
        extend(d, out=out)
        got = as_f64(out)
        assert np.isfinite(got).all()
        mine = np.zeros(76, bool)
        for a, b in zip(starts, starts[1:]):
            mine[max(0, a):max(0, b)] = True
        assert (got[~mine] == 7).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_bad_pages_are_left_out(kind, bf16):
    rng = np.random.default_rng([11, bf16])
    lengths, rows = [300, 200], [130, 3]
    d = make_rows(rng, TYPES[kind], lengths, rows, 20, 4, 2, 64, 16, bf16)
    K, V = values(d)
    table = d["table"].copy()
    bad = table.copy()
    bad[0, 3], bad[0, 12], bad[1, 0], bad[1, 12] = -1, d["n_pages"], 2 ** 31 - 1, -(2 ** 31)
    d["table"] = bad
    got = as_f64(extend(d)).reshape(-1, 4, 64)
    for s, j in [(0, 0), (0, 5), (0, 60), (0, 129), (1, 0), (1, 2)]:
        see = visible_slots(lengths[s], rows[s], j)
        see = see[np.isin(see // 16, {0: [3, 12], 1: [0, 12]}[s], invert=True)]
        for h in range(4):
            k, v = (sequence_f64(x, table[s], h // 2, lengths[s], 16)[see] for x in (K, V))
            r = int(d["starts"][s]) + j
            o, p = attend_f64(d["q"][r].reshape(4, 64)[h], k, v, 1 / 8)
            tol = 3e-2 if bf16 else 1e-4
            assert np.abs(got[r, h] - o).max() <= tol * np.abs(v).max(), (s, j, h)


@pytest.mark.parametrize("bf16", [False, True])
def test_strides_scale_and_given_output(bf16):
    rng = np.random.default_rng([12, bf16])
    d = make_rows(rng, BF16, [50, 130], [20, 130], 3, 4, 2, 64, 64, bf16)
    want, bound = extend_reference(d, 0.3)
    wide = torch.zeros((150, 1024), dtype=d["Q"].dtype, device=DEV)
    wide[:, 256:512] = d["Q"]
    d["Q"] = wide[:, 256:512]
    out = torch.full((150, 512), 7.0, dtype=wide.dtype, device=DEV)
    extend(d, out=out[:, 128:384], scale=0.3)
    check_rows(d, as_f64(out[:, 128:384].contiguous()), want, bound, "strided")
    assert (out[:, :128] == 7).all() and (out[:, 384:] == 7).all()
    for scale in (0.0, -0.2):
        got = as_f64(extend(d, scale=scale))
        w2, b2 = extend_reference(d, scale)
        check_rows(d, got, w2, np.abs(b2) + extend_reference(d, abs(scale))[1], scale)


def test_large_scores_and_small_values():
    # one slot far above the rest, then growing maxima from tile to tile
    for kind in TYPES:
        for bf16 in (False, True):
            rng = np.random.default_rng([13, bf16])
            d = make_rows(rng, TYPES[kind], [400, 260], [130, 260], 7, 4, 2, 64, 64, bf16, scale=4.0)
            run(d, scale=0.5)
            run(d, scale=4.0)
            d = make_rows(rng, TYPES[kind], [300], [140], 5, 2, 1, 64, 64, bf16, scale=1e-3)
            run(d)


@pytest.mark.parametrize("bf16", [False, True])
def test_two_streams_and_a_graph(bf16):
    rng = np.random.default_rng([14, bf16])
    d = make_rows(rng, BF16, [3000, 40, 700], [300, 3, 1], 47, 4, 2, 128, 64, bf16)
    Q, T, L, S = d["Q"], dev(d["table"]), dev(d["lengths"]), dev(d["starts"])

    def call(**kw):
        return g.gguf_attn_extend(d["cache"], Q, T, L, 3000, row_start=S, window=900, sinks=4, **kw)
    want = host(call().float())
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for s in streams:
            outs.append(call(stream=s))
    torch.cuda.synchronize()
    assert all(np.array_equal(host(o.float()), want) for o in outs)
    need = g.gguf_attn_extend_workspace(d["cache"], Q.dtype, 3, len(Q), 4, 3000, window=900, sinks=4)
    ws = torch.full((max(need, 16),), 0x7F, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(Q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(out=out, workspace=ws)
    new = torch.randn_like(Q.float()).to(Q.dtype)
    for i in range(4):
        if i == 2:   # other rows and shorter sequences under the same bound
            Q.copy_(new)
            L.copy_(dev(np.array([2000, 40, 1], np.int32)))
        want = host(call().float())
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out.float()), want), i


def test_refusals_of_the_binding():
    rng = np.random.default_rng(15)
    d = make_rows(rng, BF16, [50, 20], [3, 2], 1, 4, 2, 64, 64)
    T, L, S = dev(d["table"]), dev(d["lengths"]), dev(d["starts"])
    c, Q = d["cache"], d["Q"]
    for bad in [dict(row_start=None), dict(row_start=S[:2]), dict(row_start=S.long()), dict(out=Q[:3]),
                dict(out=torch.empty_like(Q, dtype=torch.bfloat16)), dict(workspace=torch.empty(4, device="cpu"))]:
        with pytest.raises(ValueError):
            g.gguf_attn_extend(c, Q, T, L, 64, **dict(dict(row_start=S), **bad))
    for q in (Q.half(), Q[:, :100], Q.cpu()):
        with pytest.raises(ValueError):
            g.gguf_attn_extend(c, q, T, L, 64, row_start=S)
    with pytest.raises(TypeError):
        g.gguf_attn_extend(c, None, T, L, 64)
    for bad in [dict(window=-1), dict(sinks=-1), dict(scale=math.nan), dict(out=Q), dict(max_len=-1)]:
        with pytest.raises(g.GgufQkError):
            g.gguf_attn_extend(c, Q, T, L, bad.pop("max_len", 64), row_start=S, **bad)
    empty = torch.empty((0, 256), device=DEV)
    assert g.gguf_attn_extend(c, empty, T, L, 64, row_start=torch.zeros(3, dtype=torch.int32, device=DEV)).shape == (0, 256)
