"""Inputs and bounds shared by the GPU tests of the cache, attention, eviction
and log probabilities."""

import numpy as np
import torch

import gguf_block_quant_dequant_amd as g
from oracle.formats import f32_to_bf16_bits
from oracle.serving import BF16, F16, Q8_0, attend_f64, kv_values_f64, sequence_f64

DEV = "cuda:0"
TYPES = {"f16": F16, "bf16": BF16, "q8_0": Q8_0}
U = 2.0 ** -24   # half a step of fp32, relative


def dev(a):
    return torch.from_numpy(np.array(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def cache_bytes(rng, type_id, n_pages, hkv, dim, ps, transposed, scale=1.0):
    """uint8 [n_pages, page bytes] of ordinary values."""
    shape = (n_pages, hkv, dim, ps) if transposed else (n_pages, hkv, ps, dim)
    if type_id == Q8_0:
        codes = rng.integers(-127, 128, (n_pages, hkv, ps * dim), dtype=np.int8)
        d = (scale * rng.uniform(0.005, 0.03, (n_pages, hkv, ps * dim // 32))).astype(np.float16)
        return np.concatenate([codes.view(np.uint8), d.view(np.uint8)], -1).reshape(n_pages, -1)
    x = (scale * rng.standard_normal(shape)).astype(np.float32)
    bits = x.astype(np.float16).view(np.uint16) if type_id == F16 else f32_to_bf16_bits(x)
    return np.ascontiguousarray(bits).view(np.uint8).reshape(n_pages, -1)


def poison(raw, type_id, n_pages, hkv, dim, ps, transposed, table, lengths):
    """Fills every slot that no sequence holds with NaN (Q8_0: codes of -128 with
    NaN scales), in place; raw is uint8 [n_pages, page bytes]."""
    used = np.zeros((n_pages, ps), bool)
    for row, n in zip(table, lengths):
        at = np.arange(max(0, n))
        used[row[at // ps], at % ps] = True
    heads = raw.reshape(n_pages, hkv, -1)
    n = ps * dim
    if type_id == Q8_0:
        codes, scales = heads[..., :n], heads[..., n:]
        for part, fill, per in ((codes, 0x80, dim), (scales.view(np.uint16), 0x7E00, dim // 32)):
            v = part.reshape(n_pages, hkv, per, ps) if transposed else part.reshape(n_pages, hkv, ps, per)
            v = np.moveaxis(v, 3 if transposed else 2, 1)   # [page, slot, ...]
            v[~used] = fill
            back = np.moveaxis(v, 1, 3 if transposed else 2).reshape(part.shape)
            part[...] = back
        return
    v = heads.view(np.uint16).reshape((n_pages, hkv, dim, ps) if transposed else (n_pages, hkv, ps, dim))
    np.moveaxis(v, 3 if transposed else 2, 1)[~used] = 0x7FFF


def make(rng, type_id, lengths, pages, heads, hkv, dim, ps, poisoned=True, planes=False, scale=1.0):
    """A cache for sequences of these lengths: dict of numpy arrays and the KvCache."""
    s = len(lengths)
    n_pages = s * pages + 2
    table = rng.permutation(n_pages)[:s * pages].astype(np.int32).reshape(s, pages)
    k = cache_bytes(rng, type_id, n_pages, hkv, dim, ps, False, scale)
    v = cache_bytes(rng, type_id, n_pages, hkv, dim, ps, True, scale)
    if poisoned:
        poison(k, type_id, n_pages, hkv, dim, ps, False, table, lengths)
        poison(v, type_id, n_pages, hkv, dim, ps, True, table, lengths)
    d = dict(k=k, v=v, table=table, lengths=np.asarray(lengths, np.int32), n_pages=n_pages, hkv=hkv, dim=dim, ps=ps,
             heads=heads, type=type_id, q=(2.0 * rng.standard_normal((s, heads, dim))).astype(np.float32))
    w = p = None
    if planes:
        d["weight"] = rng.uniform(0, 2, (n_pages, hkv, ps)).astype(np.float32)
        d["pos"] = np.zeros((n_pages, hkv, ps), np.int32)
        w, p = dev(d["weight"]), dev(d["pos"])
    d["cache"] = g.KvCache(dev(k), dev(v), type_id, hkv, dim, ps, weight=w, pos=p)
    return d


def values(d):
    args = (d["type"], d["n_pages"], d["hkv"], d["dim"], d["ps"])
    return kv_values_f64(d["k"], *args, False), kv_values_f64(d["v"], *args, True)


def attend_reference(d, scale, window=0, cut=None):
    """(out, error bound, weights per sequence and kv head) in fp64. The bound, per
    output: the scores' error times the softmax's sensitivity, and the sums.

    A score is a sum of dim products of a q rounded twice (scale, product: 2 U)
    and carried in parts (2^-22 at most), in fp32 (one rounding per product of
    every part, at most 3 dim): es = (2 U + 2^-22 + 3 dim U) sum|q k| scale, in
    e-folds; for Q8_0 the block sums are scaled once more (2 U). The weight's
    exponential: the difference to the maximum rounds by U of at most 2 max|s|
    log2(e), the function by 2 U, its parts carry 2^-22 (of the largest weight
    in fp16: 2^-24 2^-14 of it absolutely, below the rest). Numerator and
    denominator take this error each, and n + 64 roundings per sum of 3 n parts
    at most, and as many rescales by a rounded factor as maxima (within n)."""
    K, V = values(d)
    group = d["heads"] // d["hkv"]
    out = np.zeros((len(d["lengths"]), d["heads"], d["dim"]))
    bound = np.zeros_like(out)
    weights = []
    for s, n in enumerate(d["lengths"]):
        n = max(0, int(n)) if cut is None else max(0, min(int(n), cut))
        first = max(0, n - window) if window else 0
        per_head = []
        for h in range(d["hkv"]):
            k = sequence_f64(K, d["table"][s], h, n, d["ps"])[first:]
            v = sequence_f64(V, d["table"][s], h, n, d["ps"])[first:]
            total = np.zeros(n)
            for i in range(group):
                j = h * group + i
                q = d["q"][s, j].astype(np.float64)
                o, p = attend_f64(q, k, v, scale)
                out[s, j] = o
                if len(p):
                    total[first:] += p
                    mag = scale * (np.abs(k) @ np.abs(q))
                    es = (4 * U + 2.0 ** -22 + 3 * d["dim"] * U) * mag.max()
                    ew = es + 4 * U * mag.max() + 4 * U + 2.0 ** -22
                    bound[s, j] = (2 * ew + (8 * len(p) + 128) * U) * (p @ np.abs(v)) + 1e-30
            per_head.append(total)
        weights.append(per_head)
    return out, bound, weights


def check_bound(got, want, bound, what):
    assert np.isfinite(got).all(), what
    over = np.abs(got.astype(np.float64) - want) - bound
    assert (over <= 0).all(), (what, float(over.max()), float(np.abs(got - want).max()))
