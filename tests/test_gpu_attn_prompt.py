"""Attention of many new tokens per sequence (BF16 queries): head dims and page sizes,
bounds above the lengths, many sequences, positions split and not, the number of rows
where the kernel changes, Q8_0 scales of any size, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.serving import Q8_0, attend_f64, sequence_f64
from oracle.tokens import visible_slots
from tests.serving_util import TYPES, U, dev, values
from tests.tokens_util import BF16, HALF_BF16, HALF_F16, as_f64, check_rows, extend, extend_reference, make_rows

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def some(rows, step):
    """(sequence, row) pairs: the first and last rows, those about tiles, every step-th."""
    return {(s, j) for s, m in enumerate(rows) for j in [*range(0, m, step), 1, 31, 32, 42, 43, 63, 64, m - 2, m - 1] if 0 <= j < m}


def check(d, only, *bounds, **kw):
    """The call under each of these bounds (none: the greatest length)."""
    references = {}
    for max_len in bounds or (None,):
        cut = None if max_len is None or max_len >= d["lengths"].max() else max_len
        if cut not in references:
            references[cut] = extend_reference(d, d["dim"] ** -0.5, kw.get("window", 0), kw.get("sinks", 0), cut=cut, only=only)
        got = as_f64(extend(d, max_len=max_len, **kw))
        assert np.isfinite(got).all()
        check_rows(d, got, *references[cut], (max_len, kw))


@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_head_dims_and_bounds(kind, dim, ps):
    rng = np.random.default_rng([21, dim, ps])
    lengths, rows = [1290, 0, 90, 700], [150, 1, 90, 64]
    d = make_rows(rng, TYPES[kind], lengths, rows, -(-1290 // ps) + 3, 6, 2, dim, ps, True)
    only = some(rows, 29)
    say("prompt", kind, dim, ps)
    check(d, only, 1290, 5000, 131072, 1 << 25, 1000)
    check(d, only, 1290, 5000, 131072, 1 << 25, 1000, window=200, sinks=10)
    check(d, only, window=700, sinks=300)
    check(d, only, 131072, window=1)


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("kind", list(TYPES))
def test_pages_that_end_inside_a_tile(kind, ps):
    # lengths about the ends of pages and tiles, rows that end there
    rng = np.random.default_rng([22, ps])
    lengths = [64, 65, 63, 127, 128, 129, 144, 145, 33, 512, 513, 577]
    rows = [64, 40, 63, 100, 33, 129, 50, 145, 33, 70, 70, 70]
    d = make_rows(rng, TYPES[kind], lengths, rows, -(-577 // ps), 4, 2, 64, ps, True)
    only = some(rows, 17)
    check(d, only)
    check(d, only, window=64, sinks=16)
    check(d, only, window=63, sinks=1)
    check(d, only, window=33, sinks=128)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_more_tiles_than_blocks(kind, dim):
    # blocks enough without splitting positions
    rng = np.random.default_rng([23, dim])
    rows = rng.integers(30, 50, 130)
    lengths = rows + rng.integers(0, 100, 130)
    d = make_rows(rng, TYPES[kind], lengths, rows, 3, 8, 8, dim, 64, True)
    only = {(s, int(j)) for s, m in enumerate(rows) for j in (0, m // 2, m - 1)}
    check(d, only)
    check(d, only, window=40, sinks=3)


@pytest.mark.parametrize("dim", [64, 192])
@pytest.mark.parametrize("kind", list(TYPES))
def test_more_sequences_than_lanes_with_split_positions(kind, dim):
    rng = np.random.default_rng([24, dim])
    rows = np.full(70, 17)
    rows[[3, 69]] = 0, 90
    lengths = rows + rng.integers(0, 40, 70)
    lengths[[0, 30, 69]] = 3000, 1700, 2900
    d = make_rows(rng, TYPES[kind], lengths, rows, 47, 2, 1, dim, 64, True)
    assert g.gguf_attn_extend_workspace(d["cache"], torch.bfloat16, 70, int(rows.sum()), 2, 3000) > 0
    only = {(s, j) for s, m in enumerate(rows) for j in (0, 5, m - 1) if 0 <= j < m}
    check(d, only)
    check(d, only, 4000)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", list(TYPES))
def test_rows_about_the_change_of_kernel(kind, bf16):
    # (row, query head) pairs per sequence: 16 and 32 on average, one more, one less
    for heads, rows in ((1, [15, 15]), (1, [16, 16]), (1, [16, 17]), (1, [31, 32]), (1, [32, 32]), (1, [33, 32]), (4, [4, 4]),
                        (4, [5, 4]), (4, [8, 8]), (4, [9, 8]), (4, [1, 15]), (4, [1, 16])):
        rng = np.random.default_rng([25, heads, sum(rows)])
        d = make_rows(rng, TYPES[kind], [300, 170], rows, 5, heads, 1, 128, 64, bf16)
        check(d, None)
        check(d, None, window=100, sinks=2)


def test_bf16_rows_equal_each_other_however_they_are_grouped():
    # the same new tokens as one sequence's prompt and in two calls, the second behind the first
    rng = np.random.default_rng(26)
    for kind in TYPES:
        d = make_rows(rng, TYPES[kind], [400], [300], 7, 4, 2, 128, 64, True)
        check(d, some([300], 13))
        for a, b in ((100, 220), (220, 300)):
            part = dict(d, lengths=np.array([100 + b], np.int32), rows=[b - a], starts=np.array([0, b - a], np.int32),
                        Q=d["Q"][a:b], q=d["q"][a:b])
            check(part, some([b - a], 13))


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_drafts_under_loose_bounds(kind, dim):
    # two tiles of columns beside one read (F16 and BF16: past head dim 128 where the bound is far)
    rng = np.random.default_rng([29, dim])
    for rows in ([9, 7, 1], [1, 1, 1], [11, 0, 23]):
        d = make_rows(rng, TYPES[kind], [700, 90, 40], rows, -(-700 // 32) + 1, 6, 2, dim, 32, False)
        say("drafts", kind, dim, rows)
        check(d, None, 700, 131072, 1 << 22, 300)
        check(d, None, 700, 131072, window=100, sinks=5)
        check(d, None, 131072, window=70000, sinks=40)


PROFILES = {
    "small": lambda n, rng: 2.0 ** rng.uniform(-22, -12, n),
    "tiny": lambda n, rng: np.full(n, 2.0 ** -24),
    "large": lambda n, rng: 2.0 ** rng.uniform(8, 15.9, n),
    "rising": lambda n, rng: 2.0 ** np.linspace(-24, 15.9, n),
    "falling": lambda n, rng: 2.0 ** np.linspace(15.9, -24, n),
    "mixed": lambda n, rng: 2.0 ** rng.uniform(-24, 15.9, n),
    "zeros first": lambda n, rng: np.where(np.arange(n) < 200, 0.0, rng.uniform(0.005, 0.03, n)),
    "zeros": lambda n, rng: np.zeros(n),
    "steps": lambda n, rng: 2.0 ** np.array([-7, -8, 8, 7, -7, 9, -24])[np.arange(n) // 64 % 7],
    "one large": lambda n, rng: np.where(np.arange(n) == 150, 60000.0, 2.0 ** -10),
}


def with_scales(d, k_of, v_of, rng):
    """d with the Q8_0 scales of every held slot drawn from these profiles; their greatest."""
    ps, dim, hkv, n = d["ps"], d["dim"], d["hkv"], d["ps"] * d["dim"]
    most = []
    for name, of in (("k", k_of), ("v", v_of)):
        raw = d[name].reshape(d["n_pages"], hkv, -1).copy()
        sc = raw[..., n:].copy().view(np.float16)
        sc = sc.reshape(d["n_pages"], hkv, ps, dim // 32) if name == "k" else sc.reshape(d["n_pages"], hkv, dim // 32, ps)
        if name == "v":
            sc = sc.transpose(0, 1, 3, 2)
        top = 0.0
        for s, length in enumerate(d["lengths"]):
            at = np.arange(length)
            for h in range(hkv):
                for b in range(dim // 32):
                    x = of(length, rng).astype(np.float16)
                    sc[d["table"][s][at // ps], h, at % ps, b] = x
                    top = max(top, float(x.max()))
        if name == "v":
            sc = np.ascontiguousarray(sc.transpose(0, 1, 3, 2))
        raw[..., n:] = np.ascontiguousarray(sc).reshape(d["n_pages"], hkv, -1).view(np.uint8)
        d[name] = raw.reshape(d["n_pages"], -1)
        most.append(top)
    d["cache"] = g.KvCache(dev(d["k"]), dev(d["v"]), Q8_0, hkv, dim, ps)
    return most


@pytest.mark.parametrize("ps,dim", [(16, 64), (64, 96), (128, 128), (64, 192), (32, 256)])
@pytest.mark.parametrize("k_name,v_name", [("mixed", "rising"), ("rising", "falling"), ("falling", "mixed"), ("steps", "steps"),
                                           ("small", "large"), ("large", "small"), ("tiny", "tiny"), ("zeros", "one large"),
                                           ("one large", "zeros"), ("zeros first", "zeros first")])
def test_q8_0_scales_of_any_size(k_name, v_name, ps, dim):
    """On top of extend_reference's bound: a value whose scale is far below the tile's
    greatest is within 2^-18 of that scale (half a step of fp16's smallest numbers, 2^-25,
    in units where the greatest scale is 2^-7 or more; for a scale brought to those units
    127 + 1 such, 2^-18, where the greatest is 2^7 or more)."""
    rng = np.random.default_rng([27, ps, dim])
    lengths, rows = [700, 77], [100, 77]
    d = make_rows(rng, Q8_0, lengths, rows, -(-700 // ps), 4, 2, dim, ps, True)
    k_top, v_top = with_scales(d, PROFILES[k_name], PROFILES[v_name], rng)
    scale = 1.0 / (16 * dim ** 0.5 * max(k_top, 2.0 ** -24))
    K, V = values(d)
    got = as_f64(extend(d, scale=scale)).reshape(-1, 4, dim)
    assert np.isfinite(got).all()
    for s, j in some(rows, 31):
        r = int(d["starts"][s]) + j
        see = visible_slots(lengths[s], rows[s], j)
        for h in range(4):
            k, v = (sequence_f64(x, d["table"][s], h // 2, lengths[s], ps)[see] for x in (K, V))
            q = d["q"][r].reshape(4, dim)[h]
            o, p = attend_f64(q, k, v, scale)
            mag = scale * (np.abs(k) @ np.abs(q)).max()
            es = (4 * U + 2.0 ** -22 + HALF_F16 + 3 * dim * U) * mag + 2.0 ** -18 * scale * k_top * np.abs(q).sum()
            ew = es + 4 * U * mag + 4 * U
            bound = (2 * ew + 2.0 ** -22 + 2 * HALF_F16 + (8 * len(p) + 128) * U) * (p @ np.abs(v))
            bound += 2.0 ** -18 * v_top + 2.0 ** -25 * p.max() * np.abs(v).sum(0) + 1e-30
            bound += HALF_BF16 * (np.abs(o) + bound)
            assert (np.abs(got[r, h] - o) <= bound).all(), (s, j, h, float((np.abs(got[r, h] - o) - bound).max()))


@pytest.mark.parametrize("kind", list(TYPES))
def test_two_calls_at_once_and_replays_under_a_loose_bound(kind):
    rng = np.random.default_rng([28, len(kind)])
    d = make_rows(rng, TYPES[kind], [1500, 40, 600], [200, 40, 100], 24, 8, 2, 64, 64, True)
    T, S = dev(d["table"]), dev(d["starts"])
    L = dev(d["lengths"])

    def call(**kw):
        return g.gguf_attn_extend(d["cache"], d["Q"], T, L, 100000, row_start=S, **kw)
    want = call().float()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [call(stream=st) for _ in range(3) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o.float(), want) for o in outs)
    need = g.gguf_attn_extend_workspace(d["cache"], torch.bfloat16, 3, len(d["Q"]), 8, 100000)
    assert need > 0
    work = [torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    graphs, outs = [], []
    for ws in work:
        out, graph = torch.empty_like(d["Q"]), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call(out=out, workspace=ws)
        graphs.append(graph)
        outs.append(out)
    for lengths in ([1500, 40, 600], [700, 40, 600], [200, 40, 0], [1000, 30, 100], [1500, 40, 600]):
        L.copy_(dev(np.array(lengths, np.int32)))
        want = call().float()
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(want).all() and all(torch.equal(o.float(), want) for o in outs), lengths
