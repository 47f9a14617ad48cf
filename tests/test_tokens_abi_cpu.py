"""Refusals of the rotation, the attention of several new tokens and the
verification of drafted tokens, without a GPU: every call fails validation, or, well
formed, at the device check."""

import ctypes
import os

import pytest
import torch

import gguf_block_quant_dequant_amd as g
from gguf_block_quant_dequant_amd.build import LIB_PATH

pytestmark = [pytest.mark.skipif(not os.path.exists(LIB_PATH), reason="libgguf_qk.so not built"),
              pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="made-up device addresses: only where no GPU is visible")]

Q, K, QO, KO = 0x10000000, 0x20000000, 0x30000000, 0x38000000
FREQ, POS, AXES, NORM = 0x40000000, 0x41000000, 0x42000000, 0x43000000
TABLE, LEN, START, WS = 0x50000000, 0x51000000, 0x52000000, 0x60000000
CK, CV = 0x100000000, 0x200000000


def rope(n=8, dim=128, heads=16, kv=4, q=Q, k=K, qo=QO, ko=KO, qs=2048, ks=512, qos=2048, kos=512, type_=30, qn=NORM,
         kn=None, eps=1e-6, norms_only=False, **over):
    f = dict(freqs=FREQ, axes=AXES, pos=POS, pos_stride=8, n_axes=3, n_rot=128, pairing=1, magnitude=1.0)
    f.update(over)
    r = g.RopeStruct(**f)
    return g.lib().gguf_qk_rope(q, qs, qo, qos, heads, k, ks, ko, kos, kv, type_, n, dim, qn, kn, eps,
                                None if norms_only else ctypes.addressof(r), None)


def test_rope_refusals():
    nan, inf = float("nan"), float("inf")
    for over, status in [
            (dict(n=-1), g.ERR_SHAPE), (dict(dim=127), g.ERR_SHAPE), (dict(dim=0), g.ERR_SHAPE), (dict(dim=514), g.ERR_SHAPE),
            (dict(heads=-1), g.ERR_SHAPE), (dict(kv=-1), g.ERR_SHAPE), (dict(type_=1), g.ERR_SHAPE),
            (dict(heads=70000), g.ERR_LIMIT), (dict(q=None), g.ERR_NULL), (dict(k=None), g.ERR_NULL),
            (dict(qo=None), g.ERR_NULL), (dict(ko=None), g.ERR_NULL), (dict(eps=-1.0), g.ERR_SHAPE),
            (dict(eps=nan), g.ERR_SHAPE), (dict(eps=inf), g.ERR_SHAPE), (dict(qs=2047), g.ERR_SHAPE),
            (dict(kos=511), g.ERR_SHAPE), (dict(qs=1 << 62), g.ERR_SHAPE), (dict(n_rot=-2), g.ERR_SHAPE),
            (dict(n_rot=3), g.ERR_SHAPE), (dict(n_rot=130), g.ERR_SHAPE), (dict(n_axes=0), g.ERR_SHAPE),
            (dict(n_axes=17), g.ERR_SHAPE), (dict(pos_stride=7), g.ERR_SHAPE), (dict(pairing=2), g.ERR_SHAPE),
            (dict(magnitude=nan), g.ERR_SHAPE), (dict(magnitude=inf), g.ERR_SHAPE), (dict(pos_stride=1 << 61), g.ERR_SHAPE),
            (dict(freqs=None), g.ERR_NULL), (dict(pos=None), g.ERR_NULL), (dict(freqs=FREQ + 4), g.ERR_ALIGN),
            (dict(axes=AXES + 2), g.ERR_ALIGN), (dict(pos=POS + 1), g.ERR_ALIGN), (dict(q=Q + 1), g.ERR_ALIGN),
            (dict(ko=KO + 1), g.ERR_ALIGN), (dict(qn=NORM + 2), g.ERR_ALIGN), (dict(q=Q + 2, type_=0), g.ERR_ALIGN),
            (dict(qo=Q + 16), g.ERR_ALIAS), (dict(qo=Q, qos=4096), g.ERR_ALIAS), (dict(qo=K), g.ERR_ALIAS),
            (dict(ko=Q + 4096), g.ERR_ALIAS), (dict(ko=QO), g.ERR_ALIAS), (dict(qo=FREQ - 64), g.ERR_ALIAS),
            (dict(ko=POS), g.ERR_ALIAS), (dict(qo=AXES), g.ERR_ALIAS), (dict(qo=NORM), g.ERR_ALIAS)]:
        assert rope(**over) == status, over


def test_rope_accepts():
    for over in [dict(), dict(qo=Q, ko=K), dict(n_rot=0, freqs=None, pos=None), dict(norms_only=True), dict(axes=None),
                 dict(kv=0, k=None, ko=None), dict(heads=0, q=None, qo=None), dict(dim=2, n_rot=2), dict(q=Q + 2),
                 # q and k as slices of one product's rows, in place
                 dict(q=Q, qo=Q, k=Q + 4096, ko=Q + 4096, qs=3000, qos=3000, ks=3000, kos=3000)]:
        assert rope(**over) == g.ERR_DEVICE, over
    assert rope(n=0) == g.OK and rope(heads=0, kv=0) == g.OK
    # slices that reach into each other
    for at in (4094, 2 * 3000 - 512):
        assert rope(q=Q, qo=Q, k=Q + at, ko=Q + at, qs=3000, qos=3000, ks=3000, kos=3000) == g.ERR_ALIAS
    assert rope(q=Q, qo=Q, k=Q + 2 * 2048, ko=Q + 2 * 2048, qs=3000, qos=3000, ks=3001, kos=3001) == g.ERR_ALIAS


def cache(**over):
    f = dict(k=CK, v=CV, weight=None, pos=None, n_pages=100, type=g.TENSOR_F16, n_kv_heads=4, head_dim=128, page_size=64)
    f.update(over)
    c = g.KvCacheStruct(**f)
    c.ref = ctypes.addressof(c)
    return c


def extend(c, q=Q, type_=0, qs=2048, out=QO, os_=2048, start=START, rows=20, n=8, heads=16, table=TABLE, ts=16, lengths=LEN,
           max_len=1024, scale=0.1, window=0, sinks=0, ws=WS, wn=1 << 40):
    return g.lib().gguf_attn_extend(c.ref, q, type_, qs, out, os_, start, rows, n, heads, table, ts, lengths, max_len, scale,
                                    window, sinks, ws, wn, None)


def test_attention_refusals():
    c = cache()
    for over, status in [
            (dict(q=None), g.ERR_NULL), (dict(out=None), g.ERR_NULL), (dict(table=None), g.ERR_NULL),
            (dict(lengths=None), g.ERR_NULL), (dict(ws=None), g.ERR_NULL), (dict(type_=1), g.ERR_SHAPE),
            (dict(n=-1), g.ERR_SHAPE), (dict(rows=-1), g.ERR_SHAPE), (dict(heads=0), g.ERR_SHAPE),
            (dict(heads=6), g.ERR_SHAPE), (dict(max_len=-1), g.ERR_SHAPE), (dict(window=-1), g.ERR_SHAPE),
            (dict(sinks=-1), g.ERR_SHAPE), (dict(qs=2047), g.ERR_SHAPE), (dict(os_=2040), g.ERR_SHAPE),
            (dict(ts=0), g.ERR_SHAPE), (dict(scale=float("nan")), g.ERR_SHAPE), (dict(scale=float("inf")), g.ERR_SHAPE),
            (dict(scale=3e38), g.ERR_SHAPE), (dict(start=None), g.ERR_SHAPE), (dict(max_len=1 << 26), g.ERR_LIMIT),
            (dict(sinks=1 << 26), g.ERR_LIMIT), (dict(rows=1 << 24), g.ERR_LIMIT), (dict(n=1 << 21), g.ERR_LIMIT),
            (dict(wn=16), g.ERR_LIMIT), (dict(q=Q + 8), g.ERR_ALIGN), (dict(qs=2050), g.ERR_ALIGN),
            (dict(type_=30, os_=2052), g.ERR_ALIGN), (dict(out=QO + 8), g.ERR_ALIGN), (dict(ws=WS + 8), g.ERR_ALIGN),
            (dict(start=START + 2), g.ERR_ALIGN), (dict(lengths=LEN + 1), g.ERR_ALIGN), (dict(out=Q), g.ERR_ALIAS),
            (dict(out=Q + 64), g.ERR_ALIAS), (dict(out=CK), g.ERR_ALIAS), (dict(out=TABLE), g.ERR_ALIAS),
            (dict(out=LEN), g.ERR_ALIAS), (dict(out=START), g.ERR_ALIAS), (dict(ws=Q), g.ERR_ALIAS),
            (dict(ws=QO), g.ERR_ALIAS), (dict(ws=CV), g.ERR_ALIAS), (dict(ws=START), g.ERR_ALIAS)]:
        assert extend(c, **over) == status, over
    for type_ in (0, 30):
        for over in (dict(), dict(start=None, rows=8), dict(window=5, sinks=4), dict(window=(1 << 63) - 1),
                     dict(max_len=0), dict(sinks=1 << 25)):
            assert extend(c, type_=type_, **over) == g.ERR_DEVICE, over
    assert extend(c, n=0) == g.OK and extend(c, rows=0) == g.OK
    for over, status in [(dict(type=12), g.ERR_SHAPE), (dict(k=None), g.ERR_NULL), (dict(head_dim=80), g.ERR_SHAPE)]:
        assert extend(cache(**over)) == status
        assert g.lib().gguf_attn_extend_workspace(cache(**over).ref, 0, 1, 1, 4, 64, 0, 0) == status


def test_attention_workspace_is_what_the_call_needs():
    for kind in (1, 30, 8):
        c = cache(type=kind, page_size=16)
        for type_ in (0, 30):
            for n, rows, max_len, window, sinks in [(1, 1, 5000, 0, 0), (3, 9, 5000, 0, 0), (3, 9, 5000, 700, 4),
                                                    (2, 700, 9999, 0, 0), (1, 5000, 5000, 0, 0), (1, 64, 1 << 17, 4096, 64)]:
                need = g.lib().gguf_attn_extend_workspace(c.ref, type_, n, rows, 16, max_len, window, sinks)
                a = dict(type_=type_, n=n, rows=rows, max_len=max_len, window=window, sinks=sinks, out=1 << 40, ws=1 << 41)
                assert need >= 0 and extend(c, wn=need, **a) == g.ERR_DEVICE
                if need > 0:
                    assert extend(c, wn=need - 1, **a) == g.ERR_LIMIT
    assert g.lib().gguf_attn_extend_workspace(cache().ref, 0, 8, 16, 16, 64, 0, 0) == 0


def verify(x=CK, xs=1000, y=CV, ys=1000, type_=0, tokens=Q, u=K, un=QO, start=START, rows=20, n=4, vocab=1000, t=NORM,
           acc=POS, nxt=AXES, prob=LEN, ws=WS, wn=1 << 30):
    return g.lib().gguf_verify_draft(x, xs, y, ys, type_, tokens, u, un, start, rows, n, vocab, t, acc, nxt, prob, ws, wn, None)


def test_verify_refusals():
    for over, status in [
            (dict(x=None), g.ERR_NULL), (dict(tokens=None), g.ERR_NULL), (dict(u=None), g.ERR_NULL),
            (dict(un=None), g.ERR_NULL), (dict(start=None), g.ERR_NULL), (dict(acc=None), g.ERR_NULL),
            (dict(nxt=None), g.ERR_NULL), (dict(ws=None), g.ERR_NULL), (dict(type_=1), g.ERR_SHAPE),
            (dict(rows=-1), g.ERR_SHAPE), (dict(n=-1), g.ERR_SHAPE), (dict(vocab=0), g.ERR_SHAPE),
            (dict(xs=999), g.ERR_SHAPE), (dict(ys=999), g.ERR_SHAPE), (dict(xs=1 << 62), g.ERR_SHAPE),
            (dict(vocab=1 << 31, xs=1 << 31, ys=1 << 31), g.ERR_LIMIT), (dict(n=70000), g.ERR_LIMIT),
            (dict(rows=1 << 24), g.ERR_LIMIT), (dict(wn=64), g.ERR_LIMIT), (dict(x=CK + 2), g.ERR_ALIGN),
            (dict(y=CV + 1, type_=30), g.ERR_ALIGN), (dict(tokens=Q + 2), g.ERR_ALIGN), (dict(u=K + 1), g.ERR_ALIGN),
            (dict(ws=WS + 8), g.ERR_ALIGN), (dict(t=NORM + 2), g.ERR_ALIGN), (dict(acc=POS + 2), g.ERR_ALIGN),
            (dict(nxt=POS), g.ERR_ALIAS), (dict(prob=POS), g.ERR_ALIAS), (dict(prob=CK), g.ERR_ALIAS),
            (dict(acc=CV), g.ERR_ALIAS), (dict(ws=Q), g.ERR_ALIAS), (dict(nxt=Q), g.ERR_ALIAS), (dict(acc=START), g.ERR_ALIAS),
            (dict(acc=NORM), g.ERR_ALIAS), (dict(ws=CK), g.ERR_ALIAS)]:
        assert verify(**over) == status, over
    for over in (dict(), dict(y=None, ys=0), dict(t=None), dict(prob=None), dict(x=CK + 2, type_=30), dict(xs=1003),
                 dict(rows=0, x=None, tokens=None, u=None, y=None)):
        assert verify(**over) == g.ERR_DEVICE, over
    assert verify(n=0) == g.OK
    need = g.gguf_verify_draft_workspace(20, 4, 1000, True)
    assert need > g.gguf_verify_draft_workspace(20, 4, 1000, False) > 0
    assert verify(wn=need) == g.ERR_DEVICE and verify(wn=need - 1) == g.ERR_LIMIT


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(2, 4, 64)
    for bad in (dict(q=None, k=None), dict(q=x, k=None), dict(q=None, k=x)):
        with pytest.raises(ValueError):
            g.gguf_qk_rope(**bad)
    with pytest.raises(TypeError):
        g.gguf_qk_rope([1.0], None)
    with pytest.raises(ValueError):
        g.gguf_verify_draft(torch.zeros(2, 8), None, None, None, None)
    with pytest.raises(TypeError):
        g.gguf_verify_draft([[0.0]], None, None, None, None)
