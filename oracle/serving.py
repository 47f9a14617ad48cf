"""The steps behind the decode GEMVs (oracle; test infrastructure only): the
paged key-value cache decoded to values, the attention of one new token,
eviction by accumulated weight and the log probabilities of the head, in fp64
from the stored inputs, by plain loops over sequences and heads.

"GGUF Inferencer in R", section 5.2.1: K rows are appended per head, V is kept
transposed, attend = softmax(q k^T / sqrt(d)) v; section 5.2.3: the head's
logits become probabilities by a softmax. GGUF type ids: 1 F16, 30 BF16, 8 Q8_0.
"""

from __future__ import annotations

import numpy as np

from .formats import bf16_bits_to_f64, fp16_bits_to_f64

F16, BF16, Q8_0 = 1, 30, 8


def kv_values_f64(raw, type_id, n_pages, n_kv_heads, dim, page_size, transposed):
    """K or V pages (uint8) -> fp64 [n_pages, n_kv_heads, page_size, dim]."""
    raw = np.ascontiguousarray(raw).view(np.uint8).reshape(n_pages, n_kv_heads, -1)
    order = (dim, page_size) if transposed else (page_size, dim)
    if type_id == Q8_0:
        n = page_size * dim
        codes = raw[..., :n].view(np.int8).astype(np.float64).reshape(n_pages, n_kv_heads, *order)
        scales = fp16_bits_to_f64(np.ascontiguousarray(raw[..., n:]).view(np.uint16))
        if transposed:
            s = np.repeat(scales.reshape(n_pages, n_kv_heads, dim // 32, page_size), 32, axis=2)
        else:
            s = np.repeat(scales.reshape(n_pages, n_kv_heads, page_size, dim // 32), 32, axis=3)
        x = codes * s
    else:
        bits = raw.view(np.uint16).reshape(n_pages, n_kv_heads, *order)
        x = fp16_bits_to_f64(bits) if type_id == F16 else bf16_bits_to_f64(bits)
    return np.swapaxes(x, -1, -2) if transposed else x


def sequence_f64(pages, table_row, head, n, page_size):
    """The first n positions of one kv head of a sequence: [n, dim]."""
    at = np.arange(n)
    return pages[np.asarray(table_row)[at // page_size], head, at % page_size]


def attend_f64(q, k, v, scale):
    """softmax(scale q k^T) v of one query over [n, dim] keys and values; returns
    (out, weights). No positions: zeros."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    if len(k) == 0:
        return np.zeros(v.shape[-1] if v.ndim == 2 else len(q)), np.zeros(0)
    s = scale * (k @ q)
    e = np.exp(s - s.max())
    p = e / e.sum()
    return p @ v, p


def evict_moves(weight, pos, budget, recent):
    """(kept slots ascending, source slots, destination slots) of one kv head:
    the budget slots of greatest weight, the newest `recent` tokens above any
    weight and NaN above any number, lower slots first among equals."""
    w = np.asarray(weight, dtype=np.float64)
    n = len(w)
    if n <= budget:
        return np.arange(n), np.zeros(0, int), np.zeros(0, int)
    rank = np.zeros(n)
    rank[np.isnan(w)] = 1
    if recent:
        rank[np.asarray(pos, dtype=np.int64) > int(np.max(pos)) - recent] = 2
    value = np.where(rank > 0, 0.0, w)
    order = sorted(range(n), key=lambda i: (-rank[i], -value[i], i))
    kept = np.array(sorted(order[:budget]))
    return kept, kept[kept >= budget], np.setdiff1d(np.arange(budget), kept)


def logprobs_f64(x, tokens, top_k):
    """(log probabilities of the tokens, entropy, top ids, top log probabilities)
    of one row of logits."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        # x - max first: at magnitudes near fp32's top, max + log(sum) is max
        log_sum = np.log(np.exp(x - x.max()).sum())
        lp = (x - x.max()) - log_sum
        p = np.exp(lp)
        entropy = -np.where(p > 0, p * np.where(np.isfinite(lp), lp, 0.0), 0.0).sum()
        if np.isnan(log_sum):
            entropy = np.nan
        given = np.array([lp[t] if 0 <= t < len(x) else -np.inf for t in tokens])
    key = np.where(np.isnan(x), np.inf, x)
    order = sorted(range(len(x)), key=lambda i: (not np.isnan(x[i]), -key[i], i))[:top_k]
    return given, entropy, np.array(order, dtype=np.int64), lp[order]
