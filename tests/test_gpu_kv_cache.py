"""Appending to the paged cache and evicting from it, against the oracle: bit for
bit, with every byte outside the written slots unchanged."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.formats import f32_to_bf16_bits, quantize_q8_0_row
from oracle.serving import BF16, F16, Q8_0, evict_moves
from tests.serving_util import DEV, TYPES, cache_bytes, dev, host, make

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def views(raw, type_id, n_pages, hkv, dim, ps, transposed):
    """Writable views of cache bytes by slot: values [page, head, slot, dim] and,
    for Q8_0, scales [page, head, slot, dim / 32]."""
    heads = raw.reshape(n_pages, hkv, -1)
    n = ps * dim
    if type_id == Q8_0:
        c, s = heads[..., :n], heads[..., n:].view(np.uint16)
        if transposed:
            return (np.swapaxes(c.reshape(n_pages, hkv, dim, ps), 2, 3),
                    np.swapaxes(s.reshape(n_pages, hkv, dim // 32, ps), 2, 3))
        return c.reshape(n_pages, hkv, ps, dim), s.reshape(n_pages, hkv, ps, dim // 32)
    v = heads.view(np.uint16)
    return (np.swapaxes(v.reshape(n_pages, hkv, dim, ps), 2, 3) if transposed else v.reshape(n_pages, hkv, ps, dim),)


def stored(x, type_id):
    """A row of fp32 values as the cache stores it: (values,) or (codes, scales)."""
    if type_id == F16:
        with np.errstate(over="ignore"):
            return (x.astype(np.float16).view(np.uint16),)
    if type_id == BF16:
        return (f32_to_bf16_bits(x),)
    b = np.frombuffer(quantize_q8_0_row(x), np.uint8).reshape(-1, 34)
    return b[:, 2:].reshape(-1), np.ascontiguousarray(b[:, :2]).view(np.uint16).reshape(-1)


def append_reference(d, k, v, table, slot, seq, pos):
    kb, vb = d["k"].copy(), d["v"].copy()
    args = (d["type"], d["n_pages"], d["hkv"], d["dim"], d["ps"])
    w, p = d["weight"].copy(), d["pos"].copy()
    for x, raw, tr in ((k, kb, False), (v, vb, True)):
        parts = views(raw, *args, tr)
        for t in range(len(slot)):
            s = t if seq is None else seq[t]
            if not (0 <= s < len(table) and 0 <= slot[t] < table.shape[1] * d["ps"]):
                continue
            page = table[s, slot[t] // d["ps"]]
            if not 0 <= page < d["n_pages"]:
                continue
            i = slot[t] % d["ps"]
            for h in range(d["hkv"]):
                for part, val in zip(parts, stored(x[t].reshape(d["hkv"], d["dim"])[h], d["type"])):
                    part[page, h, i] = val
            w[page, :, i] = 0
            p[page, :, i] = slot[t] if pos is None else pos[t]
    return kb, vb, w, p


def check_append(d, k, v, table, slot, seq=None, pos=None, bf16=False, call=None):
    kb, vb, w, p = append_reference(d, k, v, table, slot, seq, pos)
    if bf16:
        dk, dv = (dev(f32_to_bf16_bits(x).view(np.int16)).view(torch.bfloat16) for x in (k, v))
    else:
        dk, dv = dev(k), dev(v)
    c = d["cache"]
    g.gguf_kv_append(c, dk, dv, dev(table), dev(slot.astype(np.int32)),
                     seq=None if seq is None else dev(seq.astype(np.int32)),
                     pos=None if pos is None else dev(pos.astype(np.int32)))
    assert np.array_equal(host(c.k), kb)
    assert np.array_equal(host(c.v), vb)
    assert np.array_equal(host(c.weight).view(np.uint32), w.view(np.uint32))
    assert np.array_equal(host(c.pos), p)


def as_bf16(x):
    return (f32_to_bf16_bits(x).astype(np.uint32) << 16).view(np.float32)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_one_token_per_sequence(kind, dim, bf16):
    rng = np.random.default_rng([dim, 1])
    d = make(rng, TYPES[kind], [0] * 11, 3, 4, 2, dim, 32, poisoned=False, planes=True)
    x = rng.standard_normal((2, 11, 2 * dim)).astype(np.float32)
    if bf16:
        x = as_bf16(x)
    say("append", kind, dim, bf16)
    check_append(d, x[0], x[1], d["table"], rng.integers(0, 96, 11), bf16=bf16)


@pytest.mark.parametrize("n,start,ps", [(1, 0, 16), (7, 0, 16), (8, 8, 16), (9, 5, 16), (64, 0, 64), (64, 3, 64),
                                        (200, 13, 32), (130, 126, 128), (1000, 24, 256)])
@pytest.mark.parametrize("kind", list(TYPES))
def test_prompt_runs_and_odd_starts(kind, n, start, ps):
    rng = np.random.default_rng([n, start])
    d = make(rng, TYPES[kind], [0, 0], -(-(start + n) // ps), 4, 3, 64, ps, poisoned=False, planes=True)
    k, v = rng.standard_normal((2, n, 3 * 64)).astype(np.float32)
    check_append(d, k, v, d["table"], start + np.arange(n), seq=np.ones(n, int), pos=np.arange(n) + 1000)


@pytest.mark.parametrize("kind", list(TYPES))
def test_mixed_sequences_scattered_slots_and_dropped_rows(kind):
    rng = np.random.default_rng(5)
    d = make(rng, TYPES[kind], [0] * 4, 4, 4, 2, 128, 32, poisoned=False, planes=True)
    n = 150
    cells = rng.permutation(4 * 128)[:n]   # no slot twice
    seq, slot = cells // 128, cells % 128
    seq[3], slot[10], seq[20], slot[30] = -1, -1, 4, 128          # padding rows, out of range
    slot[40], seq[41] = 2 ** 31 - 1, 2 ** 31 - 1
    table = d["table"].copy()
    table[2, 1], table[1, 3] = -1, d["n_pages"]                    # pages that are not there
    k, v = rng.standard_normal((2, n, 256)).astype(np.float32)
    check_append(d, k, v, table, slot, seq=seq)


def test_rounding_and_extremes():
    rng = np.random.default_rng(6)
    special = np.array([0.0, -0.0, 65504.0, 65519.9, 65520.0, -70000.0, 6e-8, 2.9e-8, 1e-30, 1.0009765, 1.0004883,
                        -1.0039063, 3.0e38, 1e-40, 127.5, -128.0], np.float32)
    for kind in TYPES:
        d = make(rng, TYPES[kind], [0], 1, 1, 1, 64, 64, poisoned=False, planes=True)
        k = rng.standard_normal((40, 64)).astype(np.float32)
        v = (k * 1e-3).astype(np.float32)
        if kind != "q8_0":
            k[0, :16], v[1, :16] = special, -special
        else:
            k[0], k[1, :32] = 0.0, 1e-9                # scales of 0 (one underflows to it)
            v[2, :32] = 127.0 * 0.5                    # ties of x / d
            v[2, 1:8] = np.array([0.25, 0.75, 1.25, -0.25, -0.75, 2.75, 63.5])
            v[3, :32] = 60000.0
        check_append(d, k, v, d["table"], np.arange(40), seq=np.zeros(40, int))


def test_append_strided_rows_without_planes_and_refusals():
    rng = np.random.default_rng(7)
    d = make(rng, TYPES["f16"], [0, 0, 0], 2, 2, 2, 64, 16, poisoned=False, planes=True)
    wide = rng.standard_normal((3, 512)).astype(np.float32)   # q | k | v rows of one buffer
    W = dev(wide)
    bare = g.KvCache(d["cache"].k, d["cache"].v, F16, 2, 64, 16)
    slot = dev(np.array([0, 17, 5], np.int32))
    g.gguf_kv_append(bare, W[:, 256:384], W[:, 384:], dev(d["table"]), slot)
    kb, vb, _, _ = append_reference(d, wide[:, 256:384], wide[:, 384:], d["table"], np.array([0, 17, 5]), None, None)
    assert np.array_equal(host(bare.k), kb) and np.array_equal(host(bare.v), vb)
    assert np.array_equal(host(d["cache"].weight), d["weight"])   # planes of another description: untouched
    t = dev(d["table"])
    with pytest.raises(ValueError):
        g.gguf_kv_append(bare, W[:, 256:384], W[:2, 384:], t, slot)
    with pytest.raises(ValueError):
        g.gguf_kv_append(bare, W[:, 256:383], W[:, 384:511], t, slot)
    with pytest.raises(ValueError):
        g.gguf_kv_append(bare, W[:, 256:384].half(), W[:, 384:].half(), t, slot)
    with pytest.raises(ValueError):
        g.gguf_kv_append(bare, W[:, 256:384], W[:, 384:], t, slot[:2])
    with pytest.raises(ValueError):
        g.gguf_kv_append(bare, W[:, 256:384], W[:, 384:], t.long(), slot)
    g.gguf_kv_append(bare, W[:0, 256:384], W[:0, 384:], t, slot[:0])
    assert np.array_equal(host(bare.k), kb)


# ------------------------------------------------------------------ eviction

def evict_reference(d, budget, recent, cut=None):
    kb, vb = d["k"].copy(), d["v"].copy()
    args = (d["type"], d["n_pages"], d["hkv"], d["dim"], d["ps"])
    parts = views(kb, *args, False) + views(vb, *args, True)
    w, p, n_out = d["weight"].copy(), d["pos"].copy(), d["lengths"].copy()
    for s, n in enumerate(d["lengths"]):
        n_out[s] = min(n, budget)
        n = min(int(n), cut) if cut else int(n)
        at = np.arange(max(n, 0))
        page, slot = d["table"][s][at // d["ps"]], at % d["ps"]
        for h in range(d["hkv"]):
            _, src, dst = evict_moves(w[page, h, slot], p[page, h, slot], budget, recent)
            for x in parts + (w, p):
                x[page[dst], h, slot[dst]] = x[page[src], h, slot[src]]
    return kb, vb, w, p, n_out


def check_evict(d, budget, recent, max_len=None, **kw):
    max_len = int(d["lengths"].max()) if max_len is None else max_len
    want = evict_reference(d, budget, recent, cut=max_len)
    c, n = d["cache"], dev(d["lengths"])
    g.gguf_kv_evict(c, dev(d["table"]), n, max_len, budget, recent=recent, **kw)
    for got, exp, what in zip((c.k, c.v, c.weight, c.pos, n), want, ("k", "v", "weight", "pos", "lengths")):
        assert np.array_equal(host(got).view(np.uint8), exp.view(np.uint8)), what


def evict_case(rng, kind, lengths, ps, hkv=2, dim=64, ties=True):
    d = make(rng, TYPES[kind], lengths, max(1, -(-max(lengths) // ps)), hkv, hkv, dim, ps, poisoned=False, planes=True)
    shape = d["weight"].shape
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if ties:
        w[rng.random(shape) < 0.2] = 0.0
        w[rng.random(shape) < 0.05] = -0.0
        w[rng.random(shape) < 0.2] = 1.5
    d["weight"] = w
    for s, n in enumerate(lengths):
        at = np.arange(n)
        for h in range(hkv):
            d["pos"][d["table"][s][at // ps], h, at % ps] = rng.permutation(n)
    d["cache"].weight.copy_(dev(w))
    d["cache"].pos.copy_(dev(d["pos"]))
    return d


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind", list(TYPES))
def test_evict_types_and_dims(kind, dim):
    rng = np.random.default_rng([dim, 2])
    say("evict", kind, dim)
    d = evict_case(rng, kind, [150, 0, 40, 41, 97], 16, dim=dim)
    check_evict(d, 40, 7)


@pytest.mark.parametrize("lengths,budget,recent", [
    ([1], 1, 1), ([2], 1, 0), ([2], 1, 1), ([33, 32, 31], 32, 0), ([33], 32, 32), ([500, 10], 499, 0), ([500], 1, 1),
    ([500], 250, 250), ([4096], 4095, 100), ([4097], 4096, 0), ([5000, 4000], 1000, 64), ([8192], 4096, 128),
    ([8193], 100, 0), ([12000, 16384], 5000, 64), ([16385], 16000, 9), ([20000], 6000, 500), ([33000], 9000, 1000), ([70000], 65000, 10)])
def test_evict_lengths(lengths, budget, recent):
    # each way of holding the keys (4, 8 and 32 per thread, and none), budgets at the edges
    rng = np.random.default_rng([lengths[0], budget])
    d = evict_case(rng, "f16", lengths, 64, hkv=1)
    check_evict(d, budget, recent)


@pytest.mark.parametrize("fill", [0.0, 1.0, np.inf, np.nan, "mixed"])
def test_evict_ties_and_special_weights(fill):
    rng = np.random.default_rng(9)
    d = evict_case(rng, "bf16", [300, 299], 32)
    if fill == "mixed":
        pick = np.array([0.0, -0.0, np.inf, -np.inf, np.nan, -1.0, 1e-45, 3e38], np.float32)
        d["weight"] = rng.choice(pick, d["weight"].shape).astype(np.float32)
    else:
        d["weight"][...] = fill
    d["cache"].weight.copy_(dev(d["weight"]))
    check_evict(d, 100, 20)


def test_evict_bound_on_the_length_and_again():
    rng = np.random.default_rng(10)
    d = evict_case(rng, "q8_0", [200, 120], 32)
    check_evict(d, 64, 8, max_len=150)   # slots behind the bound are not looked at
    d = evict_case(rng, "f16", [200, 120], 32)
    t, n = dev(d["table"]), dev(d["lengths"])
    g.gguf_kv_evict(d["cache"], t, n, 200, 64, recent=8)
    k = host(d["cache"].k)
    g.gguf_kv_evict(d["cache"], t, n, 200, 64, recent=8)   # within the budget: nothing moves
    assert np.array_equal(host(d["cache"].k), k) and host(n).tolist() == [64, 64]
    g.gguf_kv_evict(d["cache"], t, n, 20, 64, recent=8)    # a bound below the budget
    assert np.array_equal(host(d["cache"].k), k) and host(n).tolist() == [64, 64]


def test_evict_skips_bad_pages():
    rng = np.random.default_rng(21)
    d = evict_case(rng, "f16", [128], 32, hkv=1, ties=False)
    table = d["table"].copy()
    table[0, 1] = -1
    before = host(d["cache"].k), host(d["cache"].v)
    n = dev(d["lengths"])
    g.gguf_kv_evict(d["cache"], dev(table), n, 128, 64)
    assert host(n).tolist() == [64]
    # the slots of the missing page go first: every slot of the first page and
    # the 32 greatest of the last two are kept; those have nowhere to go but the
    # missing page, so nothing moves inside the cache
    w = d["weight"]
    lost = 32   # slots without a page
    kept = 64 + 0 * lost
    first = w[d["table"][0][0], 0]
    last = np.concatenate([w[d["table"][0][2], 0], w[d["table"][0][3], 0]])
    allw = np.sort(np.concatenate([first, last]))[::-1]
    floor = allw[kept - 1]
    holes = int((first < floor).sum())   # vacated slots of the first page take the first kept ones
    src = np.flatnonzero(last >= floor)[:holes]
    got = host(d["cache"].weight)[d["table"][0][0], 0]
    want = first.copy()
    want[np.flatnonzero(first < floor)] = last[src]
    assert np.array_equal(got, want)
    assert np.array_equal(host(d["cache"].k)[d["table"][0][1]], before[0][d["table"][0][1]])
    assert np.array_equal(host(d["cache"].v)[d["table"][0][1]], before[1][d["table"][0][1]])


def test_evict_in_a_graph():
    rng = np.random.default_rng(22)
    d = evict_case(rng, "bf16", [300, 180], 32)
    c, t, n = d["cache"], dev(d["table"]), dev(d["lengths"])
    start = [x.clone() for x in (c.k, c.v, c.weight, c.pos, n)]
    ws = torch.empty(g.gguf_kv_evict_workspace(c, 2, 320, 100), dtype=torch.uint8, device=DEV)
    want = evict_reference(d, 100, 10)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.gguf_kv_evict(c, t, n, 320, 100, recent=10, workspace=ws)
    for _ in range(3):
        for x, y in zip((c.k, c.v, c.weight, c.pos, n), start):
            x.copy_(y)
        torch.cuda.synchronize()
        graph.replay()
        for got, exp in zip((c.k, c.v, c.weight, c.pos, n), want):
            assert np.array_equal(host(got).view(np.uint8), exp.view(np.uint8))


def test_evict_refusals():
    rng = np.random.default_rng(23)
    d = evict_case(rng, "f16", [64], 32)
    t, n = dev(d["table"]), dev(d["lengths"])
    for kw in (dict(budget=0), dict(budget=10, recent=11), dict(budget=10, recent=-1)):
        with pytest.raises(g.GgufQkArgumentError):
            g.gguf_kv_evict(d["cache"], t, n, 64, **kw)
    bare = g.KvCache(d["cache"].k, d["cache"].v, F16, 2, 64, 32)
    with pytest.raises(g.GgufQkArgumentError):
        g.gguf_kv_evict(bare, t, n, 64, 10)
    with pytest.raises(ValueError):
        g.gguf_kv_evict(d["cache"], t, n.long(), 64, 10)
    assert host(n).tolist() == [64]


@pytest.mark.parametrize("over", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("budget", [1, 3, 16, 300, 4096, 33000])
def test_evict_few_slots_past_the_budget(budget, over):
    # a sequence that grows token by token; ties, weights of zero, holes that
    # are the newest slots themselves
    rng = np.random.default_rng([budget, over])
    d = evict_case(rng, "bf16", [budget + over, max(1, budget - 1), budget + max(1, over - 1)], 64, hkv=2)
    check_evict(d, budget, min(2, budget))
    d = evict_case(rng, "f16", [budget + over], 16, hkv=1)
    d["weight"][...] = 0.0
    d["cache"].weight.copy_(dev(d["weight"]))
    check_evict(d, budget, 0)
