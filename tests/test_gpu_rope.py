"""Norms of queries and keys per head with the rotation by position, against the fp64
oracle: types, head dims, partial rotations, pairings, axes, far positions, in place,
interleaved rows, odd alignments, streams, graphs.

Bound of an output a c - b s: the norm's factor carries the sum of dim squares (dim U),
its quotient, root and products (12 U); cosine and sine are off by the rounded fraction
of a turn (2^-26 turns, 2 pi 2^-26) and the function (2 U), together below 4 U; two
products and a sum (2 U). BF16 outputs round once more by half a step."""

import math

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.tokens import rope_f64
from tests.serving_util import DEV, U, dev, host
from tests.tokens_util import HALF_BF16, as_f64, as_type

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def reference(x, pos, freqs, axes, halves, magnitude, norm, eps, bf16):
    want = rope_f64(x, pos, freqs, axes, halves, magnitude, norm, eps)
    y = np.abs(rope_f64(x, pos, [], None, halves, 1.0, norm, eps))
    half = len(freqs)
    both = y.copy()
    for i in range(half):
        a, b = (i, i + half) if halves else (2 * i, 2 * i + 1)
        both[:, :, a] = both[:, :, b] = abs(magnitude) * (y[:, :, a] + y[:, :, b])
    bound = both * ((x.shape[-1] if norm is not None else 0) + 20) * U + 1e-37
    if bf16:
        bound += HALF_BF16 * (np.abs(want) + bound)
    return want, bound


def check(q, k, tq, tk, got, pos, freqs, axes, halves, magnitude, qn, kn, eps, bf16, what):
    for x, t, n, out in ((q, tq, qn, got[0]), (k, tk, kn, got[1])):
        want, bound = reference(x, pos, freqs, axes, halves, magnitude, n, eps, bf16)
        e = np.abs(as_f64(out).reshape(want.shape) - want) - bound
        assert (e <= 0).all(), (what, float(e.max()))


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 64), (256, 64), (96, 96), (80, 32), (128, 0), (128, 2), (64, 26), (10, 6),
                                     (2, 2), (512, 512), (510, 510), (112, 16), (24, 8)])
def test_head_dims_and_partial_rotations(dim, rot, bf16, halves):
    rng = np.random.default_rng([dim, rot, bf16, halves])
    say("rope", dim, rot, bf16, halves)
    for n, heads, kv, norms, n_axes in ((1, 4, 1, True, 1), (7, 3, 3, False, 3), (33, 7, 1, True, 2)):
        tq, q = as_type(rng.standard_normal((n, heads, dim)), bf16)
        tk, k = as_type(3 * rng.standard_normal((n, kv, dim)), bf16)
        pos = rng.integers(-50, 5000, (n_axes, n)).astype(np.int32)
        freqs = 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
        axes = rng.integers(-1, n_axes + 1, rot // 2).astype(np.int32) if n_axes > 1 else None
        qn, kn = (rng.uniform(0.5, 2, (2, dim)).astype(np.float32)) if norms else (None, None)
        if n == 33:
            kn = None   # keys not normed
        mag = 1.0 if n == 1 else 1.3
        f = torch.tensor(freqs, dtype=torch.float64, device=DEV) if rot else None
        if rot == 0:
            axes, n_axes = None, 1
        got = g.gguf_qk_rope(tq, tk, None if f is None else dev(pos if n_axes > 1 else pos[0]), f,
                             None if axes is None else dev(axes), halves=halves, magnitude=mag,
                             q_norm=None if qn is None else dev(qn), k_norm=None if kn is None else dev(kn), eps=1e-5)
        check(q, k, tq, tk, got, pos, freqs, axes, halves, mag, qn, kn, 1e-5, bf16, (dim, rot, n))


@pytest.mark.parametrize("bf16", [False, True])
def test_far_positions_keep_their_angle(bf16):
    rng = np.random.default_rng(2)
    pos = np.array([[0, 1, 131071, 1000003, 2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 7]], np.int32)
    freqs = 500000.0 ** (-np.arange(64) / 64)
    tq, q = as_type(rng.standard_normal((7, 5, 128)), bf16)
    tk, k = as_type(rng.standard_normal((7, 2, 128)), bf16)
    got = g.gguf_qk_rope(tq, tk, dev(pos[0]), torch.tensor(freqs, device=DEV))
    # fp64 turns: 2^31 radians to 2^-52 of them add 2^-21 of a radian
    for x, out in ((q, got[0]), (k, got[1])):
        want, bound = reference(x, pos, freqs, None, True, 1.0, None, 0, bf16)
        near = np.abs(as_f64(out) - want) - bound
        assert (near[[0, 1, 2, 3]] <= 0).all()
        assert (near <= 2.0 ** -20 * np.abs(x).max() * 2).all()


@pytest.mark.parametrize("bf16", [False, True])
def test_in_place_and_slices_of_one_product(bf16):
    rng = np.random.default_rng(3)
    n, heads, kv, dim = 37, 6, 2, 64
    row = (heads + 2 * kv) * dim
    for pad in (0, 8, 3):   # 3: rows that are not 16-byte aligned
        buf, x = as_type(rng.standard_normal((n, row + pad)), bf16)
        keep = as_f64(buf)
        q, k = buf[:, :heads * dim].unflatten(1, (heads, dim)), buf[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim))
        pos, freqs = rng.integers(0, 999, (1, n)).astype(np.int32), 100.0 ** (-np.arange(32) / 32)
        w = rng.uniform(0.5, 2, dim).astype(np.float32)
        qx, kx = x[:, :heads * dim].reshape(n, heads, dim), x[:, heads * dim:(heads + kv) * dim].reshape(n, kv, dim)
        out = g.gguf_qk_rope(q, k, dev(pos[0]), torch.tensor(freqs, device=DEV), q_norm=dev(w), q_out=q, k_out=k)
        assert out[0].data_ptr() == q.data_ptr()
        got = as_f64(buf)
        for a, b, xx, nn in ((0, heads, qx, w), (heads, heads + kv, kx, None)):
            want, bound = reference(xx, pos, freqs, None, True, 1.0, nn, 1e-6, bf16)
            assert (np.abs(got[:, a * dim:b * dim].reshape(want.shape) - want) <= bound).all(), pad
        rest = slice((heads + kv) * dim, None)
        assert np.array_equal(got[:, rest], keep[:, rest])   # v and the padding stay


@pytest.mark.parametrize("bf16", [False, True])
def test_one_side_alone_and_norms_alone(bf16):
    rng = np.random.default_rng(4)
    tx, x = as_type(rng.standard_normal((9, 4, 96)), bf16)
    w = rng.uniform(0.5, 2, 96).astype(np.float32)
    pos, freqs = np.arange(9, dtype=np.int32)[None], 10.0 ** (-np.arange(48) / 48)
    f = torch.tensor(freqs, device=DEV)
    a, none = g.gguf_qk_rope(tx, None, dev(pos[0]), f)
    none2, b = g.gguf_qk_rope(None, tx, dev(pos[0]), f)
    assert none is None and none2 is None and np.array_equal(as_f64(a), as_f64(b))
    got, _ = g.gguf_qk_rope(tx, None, q_norm=dev(w), eps=0.5)
    want, bound = reference(x, pos, [], None, True, 1.0, w, 0.5, bf16)
    assert (np.abs(as_f64(got) - want) <= bound).all()
    zero = torch.zeros_like(tx)
    assert not as_f64(g.gguf_qk_rope(zero, None, q_norm=dev(w), eps=1e-6)[0]).any()


@pytest.mark.parametrize("tokens", [1, 2, 2047, 2049, 4099, 16385, 20001])
def test_many_tokens(tokens):
    # block sizes change with the number of tokens: every token is written
    rng = np.random.default_rng(tokens)
    x = rng.standard_normal((tokens, 2, 64)).astype(np.float32)
    y = rng.standard_normal((tokens, 1, 64)).astype(np.float32)
    pos = rng.integers(0, 100000, (1, tokens)).astype(np.int32)
    freqs = 1000.0 ** (-np.arange(32) / 32)
    tq, tk = dev(x), dev(y)
    got = g.gguf_qk_rope(tq, tk, dev(pos[0]), torch.tensor(freqs, device=DEV), q_out=torch.full_like(tq, 9.0))
    at = np.unique(np.concatenate([np.arange(min(9, tokens)), rng.integers(0, tokens, 60), [tokens - 1]]))
    for v, o in ((x, got[0]), (y, got[1])):
        want, bound = reference(v[at].astype(np.float64), pos[:, at], freqs, None, True, 1.0, None, 0, False)
        assert (np.abs(as_f64(o)[at] - want) <= bound).all()
        # turning keeps every pair's length
        h = host(o)
        assert np.allclose((h ** 2).sum(-1), (v ** 2).sum(-1), rtol=1e-5)


def test_stream_and_graph():
    rng = np.random.default_rng(6)
    tq, _ = as_type(rng.standard_normal((40, 8, 128)), True)
    tk, _ = as_type(rng.standard_normal((40, 2, 128)), True)
    pos = dev(np.arange(40, dtype=np.int32))
    f = torch.tensor(500000.0 ** (-np.arange(64) / 64), device=DEV)
    w = dev(rng.uniform(0.5, 2, 128).astype(np.float32))
    want = [as_f64(o) for o in g.gguf_qk_rope(tq, tk, pos, f, q_norm=w, k_norm=w)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = g.gguf_qk_rope(tq, tk, pos, f, q_norm=w, k_norm=w, stream=s)
    torch.cuda.synchronize()
    assert all(np.array_equal(as_f64(o), w_) for o, w_ in zip(out, want))
    qo, ko = torch.empty_like(tq), torch.empty_like(tk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gguf_qk_rope(tq, tk, pos, f, q_norm=w, k_norm=w, q_out=qo, k_out=ko)
    for i in range(3):
        pos += 1000
        want = [as_f64(o) for o in g.gguf_qk_rope(tq, tk, pos, f, q_norm=w, k_norm=w)]
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(as_f64(qo), want[0]) and np.array_equal(as_f64(ko), want[1]), i


def test_refusals_of_the_binding():
    x = torch.zeros((4, 2, 64), device=DEV)
    pos, f = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(32, dtype=torch.float64, device=DEV)
    for bad in [dict(k=x.bfloat16()), dict(k=x[:3]), dict(k=x[:, :, :32]), dict(pos=pos[:3]), dict(pos=pos.long()),
                dict(pos=None), dict(freqs=None), dict(freqs=f.float()), dict(axes=pos), dict(q_norm=f.float()),
                dict(q_out=x[:2]), dict(k_out=torch.zeros_like(x, dtype=torch.bfloat16)), dict(q=x.half()),
                dict(q=x.view(4, 128)), dict(q=x.transpose(1, 2)), dict(freqs=torch.zeros(33, dtype=torch.float64, device=DEV))]:
        with pytest.raises(ValueError):
            g.gguf_qk_rope(**dict(dict(q=x, k=x.clone(), pos=pos, freqs=f), **bad))
    with pytest.raises(g.GgufQkError):
        g.gguf_qk_rope(x, x, pos, f, q_out=x, k_out=x)
    with pytest.raises(g.GgufQkError):
        g.gguf_qk_rope(x, None, pos, f, magnitude=math.inf)
    empty = torch.zeros((0, 2, 64), device=DEV)
    assert g.gguf_qk_rope(empty, None, pos[:0], f)[0].shape == (0, 2, 64)
