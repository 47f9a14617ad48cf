"""Inputs, references and bounds shared by the GPU tests of the operators over several
new tokens."""

import numpy as np
import torch

import gguf_block_quant_dequant_amd as g
from oracle.formats import bf16_bits_to_f64, f32_to_bf16_bits
from oracle.serving import BF16, F16, Q8_0, attend_f64, sequence_f64
from oracle.tokens import visible_slots
from tests.serving_util import U, dev, host, make, values

HALF_BF16, HALF_F16 = 2.0 ** -8, 2.0 ** -11   # half a step, relative


def as_type(x, bf16):
    """A device tensor of the values rounded to the type, and the values as fp64."""
    x = np.asarray(x, np.float32)
    if not bf16:
        return dev(x), x.astype(np.float64)
    bits = f32_to_bf16_bits(x)
    return dev(bits.view(np.int16)).view(torch.bfloat16), bf16_bits_to_f64(bits)


def as_f64(t):
    if t.dtype is torch.bfloat16:
        return bf16_bits_to_f64(host(t.view(torch.int16)).view(np.uint16))
    return host(t).astype(np.float64)


def make_rows(rng, type_id, lengths, rows, pages, heads, hkv, dim, ps, bf16=False, scale=1.0, extra=0):
    """A cache for sequences of these lengths whose newest rows[s] tokens have queries,
    and `extra` rows of q behind them that belong to no sequence."""
    d = make(rng, type_id, lengths, pages, heads, hkv, dim, ps, scale=scale)
    n = int(sum(rows))
    d["rows"], d["starts"] = list(rows), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    d["bf16"] = bf16
    d["Q"], d["q"] = as_type(2.0 * rng.standard_normal((n + extra, heads * dim)), bf16)
    return d


def extend(d, max_len=None, starts=True, **kw):
    n = int(max(d["lengths"].max(), 1)) if max_len is None else max_len
    return g.gguf_attn_extend(d["cache"], d["Q"], dev(d["table"]), dev(d["lengths"]), n,
                              row_start=dev(d["starts"]) if starts else None, **kw)


def extend_reference(d, scale, window=0, sinks=0, cut=None, only=None):
    """(out, bound) in fp64, rows [n, heads, dim]; `only`: the (sequence, row) pairs to
    compute (others are NaN).

    The bound, per output. A score is a sum of dim products: operands in parts (2^-22 of
    q, as in gguf_attn_decode) or exact, Q8_0 keys past that rounded to fp16 (half a
    step) in BF16 calls; one rounding per product (3 dim U). es = that, times
    scale sum|q k|, in e-folds. The exponential's argument rounds by 2 U of the greatest
    score's magnitude, twice; the function by 2 U. In BF16 calls a weight may be rounded
    to the operand type: half a step of bf16 or fp16, or half a step of fp16's smallest
    numbers (2^-25) of the greatest weight; Q8_0 values to fp16. Sums: n + 64 roundings
    and as many rescales. The output rounds by half a step of its type. In F32 calls a
    weight is two fp16 after a factor 2^14, so that what the second cannot hold, half a
    step of its smallest numbers, is 2^-25 2^-14 = 2^-39 of the greatest weight: it counts
    where a slot of tiny values holds nearly all the weight. Q8_0 takes that of the weight
    times the scale, of the greatest scale met, 127 codes of which bound a value."""
    K, V = values(d)
    group = d["heads"] // d["hkv"]
    n_rows = len(d["q"])
    out = np.full((n_rows, d["heads"], d["dim"]), np.nan)
    bound = np.zeros_like(out)
    bf16 = d["bf16"]
    kq = 2.0 ** -22 + (HALF_F16 if bf16 and d["type"] == Q8_0 else 0.0)
    wq = 2.0 ** -22
    tiny = 0.0 if d["type"] == BF16 else 2.0 ** -39
    if bf16:
        wq += HALF_BF16 if d["type"] == BF16 else HALF_F16
        wq += HALF_F16 if d["type"] == Q8_0 else 0.0
        tiny = 0.0 if d["type"] == BF16 else 2.0 ** -25
    for s, (length, m) in enumerate(zip(d["lengths"], d["rows"])):
        held = max(0, int(length))
        held = held if cut is None else min(held, cut)
        for h in range(d["hkv"]):
            k = sequence_f64(K, d["table"][s], h, held, d["ps"])
            v = sequence_f64(V, d["table"][s], h, held, d["ps"])
            top = 127 * np.nanmax(np.abs(v)) if held else 0.0   # a code is at least 1 where a value is not 0
            for j in range(m):
                if only is not None and (s, j) not in only:
                    continue
                r = int(d["starts"][s]) + j
                see = visible_slots(held, m, j, window, sinks)
                kk, vv = k[see], v[see]
                for i in range(group):
                    q = d["q"][r].reshape(d["heads"], d["dim"])[h * group + i]
                    o, p = attend_f64(q, kk, vv, scale)
                    out[r, h * group + i] = o
                    if len(p):
                        few = np.abs(vv).sum(0)
                        if d["type"] == Q8_0 and not bf16:
                            few = few + len(p) * top
                        mag = (scale * (np.abs(kk) @ np.abs(q))).max()
                        es = (4 * U + kq + 3 * d["dim"] * U) * mag
                        ew = es + 4 * U * mag + 4 * U
                        bound[r, h * group + i] = ((2 * ew + wq + (8 * len(p) + 128) * U) * (p @ np.abs(vv))
                                                   + tiny * p.max() * few + 1e-30)
    if bf16:
        bound += HALF_BF16 * (np.abs(out) + bound)
    return out, bound


def check_rows(d, got, want, bound, what):
    """Rows of `got` (of every sequence's rows) within the bound."""
    got = got.reshape(want.shape)
    done = ~np.isnan(want)
    assert np.isfinite(got[done]).all(), what
    over = np.abs(got - want)[done] - bound[done]
    assert (over <= 0).all(), (what, float(over.max()), float(np.abs(got - want)[done].max()))


__all__ = ["BF16", "F16", "Q8_0", "U", "as_f64", "as_type", "check_rows", "dev", "extend", "extend_reference", "host",
           "make_rows"]
