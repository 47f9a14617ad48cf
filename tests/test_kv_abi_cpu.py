"""Refusals of the cache, attention, eviction and log probability entry points,
without a GPU: every call fails validation, or, well formed, at the device check."""

import ctypes
import os

import pytest
import torch

import gguf_block_quant_dequant_amd as g
from gguf_block_quant_dequant_amd.build import LIB_PATH

pytestmark = [pytest.mark.skipif(not os.path.exists(LIB_PATH), reason="libgguf_qk.so not built"),
              pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="made-up device addresses: only where no GPU is visible")]

K, V, W, P = 0x10000000, 0x20000000, 0x30000000, 0x38000000
Q, OUT, TABLE, LEN, WS = 0x40000000, 0x48000000, 0x50000000, 0x51000000, 0x60000000


def cache(**over):
    f = dict(k=K, v=V, weight=W, pos=P, n_pages=100, type=g.TENSOR_F16, n_kv_heads=4, head_dim=128, page_size=64)
    f.update(over)
    c = g.KvCacheStruct(**f)
    c.ref = ctypes.addressof(c)
    return c


BAD_CACHES = [
    (dict(k=None), g.ERR_NULL), (dict(v=None), g.ERR_NULL), (dict(type=12), g.ERR_SHAPE), (dict(type=0), g.ERR_SHAPE),
    (dict(head_dim=80), g.ERR_SHAPE), (dict(head_dim=0), g.ERR_SHAPE), (dict(head_dim=512), g.ERR_SHAPE),
    (dict(page_size=8), g.ERR_SHAPE), (dict(page_size=48), g.ERR_SHAPE), (dict(page_size=512), g.ERR_SHAPE),
    (dict(page_size=-16), g.ERR_SHAPE), (dict(n_kv_heads=0), g.ERR_SHAPE), (dict(n_kv_heads=-1), g.ERR_SHAPE),
    (dict(n_kv_heads=70000), g.ERR_LIMIT), (dict(n_pages=0), g.ERR_SHAPE), (dict(n_pages=1 << 40), g.ERR_SHAPE),
    (dict(k=K + 8), g.ERR_ALIGN), (dict(v=V + 2), g.ERR_ALIGN), (dict(weight=W + 4), g.ERR_ALIGN),
    (dict(pos=P + 4), g.ERR_ALIGN), (dict(v=K), g.ERR_ALIAS), (dict(weight=K + 1024), g.ERR_ALIAS),
    (dict(pos=W), g.ERR_ALIAS),
]


def append(c, k=Q, v=OUT, src=0, stride=512, n=8, seq=None, slot=LEN, pos=None, table=TABLE, ts=16, ns=8):
    return g.lib().gguf_kv_append(c.ref, k, v, src, stride, n, seq, slot, pos, table, ts, ns, None)


def attend(c, q=Q, qs=2048, out=OUT, os_=2048, n=8, heads=16, table=TABLE, ts=16, lengths=LEN, max_len=1024, scale=0.1,
           window=0, track=0, ws=WS, wn=1 << 40):
    return g.lib().gguf_attn_decode(c.ref, q, qs, out, os_, n, heads, table, ts, lengths, max_len, scale, window,
                                    track, ws, wn, None)


def evict(c, n=8, table=TABLE, ts=16, lengths=LEN, max_len=1024, budget=512, recent=16, ws=WS, wn=1 << 40):
    return g.lib().gguf_kv_evict(c.ref, n, table, ts, lengths, max_len, budget, recent, ws, wn, None)


def logprobs(x=K, type_=0, n=4, vocab=1000, stride=1000, tokens=LEN, nt=2, k=5, lp=Q, ent=OUT, ids=TABLE, top=V, ws=WS,
             wn=1 << 40):
    return g.lib().gguf_logprobs(x, type_, n, vocab, stride, tokens, nt, k, lp, ent, ids, top, ws, wn, None)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_cache_description(over, status):
    c = cache(**over)
    for call in (append, attend, evict):
        assert call(c) == status
    assert g.lib().gguf_attn_decode_workspace(c.ref, 1, 4, 64, 0) == status
    assert g.lib().gguf_kv_evict_workspace(c.ref, 1, 64, 32) == status


def test_null_cache_and_well_formed_calls():
    class Null:
        ref = None
    for call in (append, attend, evict):
        assert call(Null) == g.ERR_NULL
        assert call(cache()) == g.ERR_DEVICE   # accepted: only the device is missing
    assert logprobs() == g.ERR_DEVICE


def test_page_bytes():
    assert g.gguf_kv_page_bytes(g.TENSOR_F16, 4, 128, 64) == 4 * 128 * 64 * 2
    assert g.gguf_kv_page_bytes(g.TENSOR_BF16, 1, 64, 16) == 2048
    assert g.gguf_kv_page_bytes(g.TYPE_Q8_0, 4, 128, 64) == 4 * 64 * 136
    for bad in ((12, 4, 128, 64), (1, 0, 128, 64), (1, 4, 100, 64), (1, 4, 128, 24), (1, 1 << 60, 256, 256)):
        assert g.gguf_kv_page_bytes(*bad) == g.ERR_SHAPE


def test_append_refusals():
    c = cache()
    for over, status in [(dict(k=None), g.ERR_NULL), (dict(v=None), g.ERR_NULL), (dict(slot=None), g.ERR_NULL),
                         (dict(table=None), g.ERR_NULL), (dict(src=1), g.ERR_SHAPE), (dict(stride=511), g.ERR_SHAPE),
                         (dict(n=-1), g.ERR_SHAPE), (dict(ns=-1), g.ERR_SHAPE), (dict(ts=0), g.ERR_SHAPE),
                         (dict(stride=513), g.ERR_ALIGN), (dict(k=Q + 4), g.ERR_ALIGN), (dict(slot=LEN + 2), g.ERR_ALIGN),
                         (dict(seq=TABLE + 1), g.ERR_ALIGN), (dict(n=1 << 60), g.ERR_SHAPE), (dict(k=K), g.ERR_ALIAS),
                         (dict(v=V + 4096), g.ERR_ALIAS), (dict(slot=W), g.ERR_ALIAS), (dict(table=P), g.ERR_ALIAS)]:
        assert append(c, **over) == status, over
    assert append(c, n=0) == g.OK


def test_attention_refusals():
    c = cache()
    for over, status in [(dict(q=None), g.ERR_NULL), (dict(out=None), g.ERR_NULL), (dict(table=None), g.ERR_NULL),
                         (dict(lengths=None), g.ERR_NULL), (dict(ws=None), g.ERR_NULL), (dict(n=-1), g.ERR_SHAPE),
                         (dict(heads=0), g.ERR_SHAPE), (dict(heads=6), g.ERR_SHAPE), (dict(max_len=-1), g.ERR_SHAPE),
                         (dict(window=-1), g.ERR_SHAPE), (dict(qs=2047), g.ERR_SHAPE), (dict(os_=4), g.ERR_SHAPE),
                         (dict(ts=0), g.ERR_SHAPE), (dict(scale=float("nan")), g.ERR_SHAPE),
                         (dict(scale=float("inf")), g.ERR_SHAPE), (dict(n=70000), g.ERR_LIMIT),
                         (dict(heads=1 << 20, qs=1 << 27, os_=1 << 27), g.ERR_LIMIT), (dict(max_len=1 << 31), g.ERR_LIMIT),
                         (dict(wn=16), g.ERR_LIMIT), (dict(q=Q + 4), g.ERR_ALIGN), (dict(qs=2050), g.ERR_ALIGN),
                         (dict(out=OUT + 8), g.ERR_ALIGN), (dict(ws=WS + 4), g.ERR_ALIGN),
                         (dict(lengths=LEN + 2), g.ERR_ALIGN), (dict(out=Q), g.ERR_ALIAS), (dict(out=Q + 16), g.ERR_ALIAS),
                         (dict(out=K + 64), g.ERR_ALIAS), (dict(ws=V), g.ERR_ALIAS), (dict(ws=Q), g.ERR_ALIAS),
                         (dict(out=TABLE), g.ERR_ALIAS), (dict(track=1, q=W), g.ERR_ALIAS),
                         (dict(track=1, lengths=W), g.ERR_ALIAS)]:
        assert attend(c, **over) == status, over
    assert attend(cache(weight=None), track=1) == g.ERR_NULL
    assert attend(cache(weight=None)) == g.ERR_DEVICE
    assert attend(c, n=0) == g.OK
    # rows that fit one split need no workspace
    assert g.lib().gguf_attn_decode_workspace(c.ref, 8, 16, 64, 0) == 0
    assert attend(c, max_len=64, ws=None, wn=0) == g.ERR_DEVICE


def test_attention_workspace_covers_every_window():
    # a window may cut the positions into other chunks: never more bytes
    c = cache(page_size=16)
    for n, max_len in ((1, 2000), (3, 5000), (1, 4097), (40, 3000), (7, 9999)):
        need = g.lib().gguf_attn_decode_workspace(c.ref, n, 16, max_len, 0)
        for window in [0, 1, 31, 500, 1790, 1900, max_len - 1, max_len, max_len + 5] + list(range(100, max_len, 371)):
            assert attend(c, n=n, max_len=max_len, window=window, wn=need) == g.ERR_DEVICE, (n, max_len, window)


def test_eviction_refusals():
    c = cache()
    for over, status in [(dict(table=None), g.ERR_NULL), (dict(lengths=None), g.ERR_NULL), (dict(ws=None), g.ERR_NULL),
                         (dict(n=-1), g.ERR_SHAPE), (dict(budget=0), g.ERR_SHAPE), (dict(recent=-1), g.ERR_SHAPE),
                         (dict(recent=513), g.ERR_SHAPE), (dict(max_len=-1), g.ERR_SHAPE), (dict(ts=0), g.ERR_SHAPE),
                         (dict(n=70000), g.ERR_LIMIT), (dict(max_len=1 << 31), g.ERR_LIMIT), (dict(wn=16), g.ERR_LIMIT),
                         (dict(ws=WS + 8), g.ERR_ALIGN), (dict(lengths=LEN + 1), g.ERR_ALIGN),
                         (dict(lengths=W), g.ERR_ALIAS), (dict(ws=K), g.ERR_ALIAS), (dict(ws=TABLE), g.ERR_ALIAS),
                         (dict(lengths=TABLE), g.ERR_ALIAS)]:
        assert evict(c, **over) == status, over
    assert evict(cache(weight=None)) == g.ERR_NULL
    assert evict(cache(pos=None)) == g.ERR_NULL
    assert evict(cache(pos=None), recent=0) == g.ERR_DEVICE
    assert evict(c, n=0) == g.OK
    assert evict(c, max_len=512, ws=None, wn=0) == g.ERR_DEVICE   # nothing can exceed the budget


def test_logprobs_refusals():
    for over, status in [(dict(x=None), g.ERR_NULL), (dict(tokens=None), g.ERR_NULL), (dict(lp=None), g.ERR_NULL),
                         (dict(ids=None), g.ERR_NULL), (dict(top=None), g.ERR_NULL), (dict(type_=1), g.ERR_SHAPE),
                         (dict(n=-1), g.ERR_SHAPE), (dict(vocab=0), g.ERR_SHAPE), (dict(stride=999), g.ERR_SHAPE),
                         (dict(k=-1), g.ERR_SHAPE), (dict(vocab=4, stride=4), g.ERR_SHAPE), (dict(nt=-1), g.ERR_SHAPE),
                         (dict(k=65), g.ERR_LIMIT), (dict(vocab=1 << 31, stride=1 << 31), g.ERR_LIMIT),
                         (dict(vocab=20000, stride=20000, wn=64), g.ERR_LIMIT),
                         (dict(vocab=20000, stride=20000, ws=None), g.ERR_NULL), (dict(x=K + 2), g.ERR_ALIGN),
                         (dict(x=K + 1, type_=30), g.ERR_ALIGN), (dict(lp=Q + 2), g.ERR_ALIGN), (dict(lp=K), g.ERR_ALIAS),
                         (dict(ent=Q), g.ERR_ALIAS), (dict(top=TABLE), g.ERR_ALIAS),
                         (dict(vocab=20000, stride=20000, ws=Q), g.ERR_ALIAS)]:
        assert logprobs(**over) == status, over
    assert logprobs(n=0) == g.OK
    assert logprobs(tokens=None, lp=None, nt=0, ids=None, top=None, k=0, ent=None) == g.ERR_DEVICE
    assert g.gguf_logprobs_workspace(4, 1000, 5) == 0 and g.gguf_logprobs_workspace(4, 128256, 5) > 0
    assert g.gguf_logprobs_workspace(4, 10, 11) == g.ERR_SHAPE


def test_binding_refuses_host_tensors_and_shapes():
    with pytest.raises(ValueError):
        g.KvCache(torch.zeros(16384, dtype=torch.uint8), torch.zeros(16384, dtype=torch.uint8), g.TENSOR_F16, 1, 64, 16)
    with pytest.raises(ValueError):
        g.KvCache(None, None, g.TYPE_Q4_K, 1, 64, 16)
    with pytest.raises(ValueError):
        g.gguf_logprobs(torch.zeros(2, 8))
    with pytest.raises(TypeError):
        g.gguf_logprobs([0.0, 1.0])
