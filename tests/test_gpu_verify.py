"""Verification of drafted tokens against the fp64 oracle: types, vocabularies from one
to long ones, ragged rows, temperatures with 0, drafts without probabilities, ruled-out
tokens, rows without a distribution, tokens outside, borders, strides, streams, graphs.

Tokens and counts have to be equal: sums are fp64 on both sides, so that they could
differ only where a number falls within about 1e-12 of a border. accept_prob is a
quotient of fp64 values rounded once to fp32 (U); its sums add 2^-40."""

import numpy as np
import pytest
import torch

import gguf_block_quant_dequant_amd as g
from oracle.tokens import softmax_f64, verify_f64
from tests.serving_util import DEV, U, dev, host
from tests.tokens_util import as_type

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


def batch(rng, rows, vocab, bf16, noise=0.7, ruled_out=True):
    n = int(sum(rows))
    x = 2.0 * rng.standard_normal((n, vocab))
    if vocab > 40:
        x[np.arange(n)[:, None], rng.integers(0, vocab, (n, 8))] += rng.uniform(0, 8, (n, 8))
    y = x + noise * rng.standard_normal((n, vocab))
    if ruled_out and vocab > 4:
        x[:, rng.integers(0, vocab, vocab // 5)] = -np.inf
        y[:, rng.integers(0, vocab, vocab // 5)] = -np.inf
    tx, x = as_type(x, bf16)
    ty, y = as_type(y, bf16)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    tokens = np.array([rng.choice(vocab, p=softmax_f64(r)) if vocab > 1 else 0 for r in y], np.int32).reshape(n)
    return dict(tx=tx, ty=ty, x=x, y=y, starts=starts, tokens=tokens, u=rng.random(n).astype(np.float32),
                un=rng.random(len(rows)).astype(np.float32), t=None)


def check(b, draft=True, **kw):
    t = None if b["t"] is None else dev(b["t"])
    r = g.gguf_verify_draft(b["tx"], dev(b["tokens"]), dev(b["u"]), dev(b["un"]), dev(b["starts"]),
                            draft=b["ty"] if draft else None, temperature=t, **kw)
    acc, nxt, prob = verify_f64(b["x"], b["y"] if draft else None, b["tokens"], b["u"], b["un"], b["starts"], b["t"])
    assert np.array_equal(host(r.accepted), acc) and np.array_equal(host(r.next_tokens), nxt)
    mine = ~np.isnan(prob)
    assert np.allclose(host(r.accept_prob)[mine], prob[mine], rtol=2 * U, atol=1e-37)
    return acc, nxt


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 5, 255, 997, 4096, 8191, 8192, 8193, 16390, 32000, 50257])
def test_vocabularies(vocab, bf16):
    rng = np.random.default_rng([vocab, bf16])
    say("verify", vocab, bf16)
    for draft in (True, False):
        b = batch(rng, [4, 1, 6, 2, 5], vocab, bf16)
        check(b, draft)
        b["t"] = np.array([0.7, 0.0, 1.5, 0.0, 0.05], np.float32)
        check(b, draft)


def test_every_length_is_met():
    # enough sequences for each number of accepted tokens, and both ways to end
    rng = np.random.default_rng(1)
    b = batch(rng, [5] * 90, 700, False, noise=0.3)
    acc, _ = check(b)
    assert set(acc.tolist()) == {0, 1, 2, 3, 4}
    # equal probabilities: all accepted but tokens that are ruled out, after which
    # nothing is left of p - q and p is drawn from
    b["ty"], b["y"] = b["tx"], b["x"]
    acc, _ = check(b)
    out = np.isinf(b["x"][np.arange(450), b["tokens"]]).reshape(90, 5)
    out[:, 4] = True
    assert np.array_equal(acc, out.argmax(1))


def test_long_vocabulary():
    rng = np.random.default_rng(2)
    for bf16 in (False, True):
        b = batch(rng, [5, 3, 9, 1], 128256, bf16)
        b["t"] = np.array([0.8, 1.2, 0.6, 1.0], np.float32)
        check(b)
        check(b, draft=False)


def test_many_draws_from_flat_rows():
    # flat rows put a border every 1 / vocab: sums in fp32 would miss some of them
    rng = np.random.default_rng(3)
    b = batch(rng, [1] * 300, 30011, False, ruled_out=False)
    b["x"] *= 0.01
    b["tx"] = dev(b["x"].astype(np.float32))
    b["x"] = b["x"].astype(np.float32).astype(np.float64)
    check(b)


@pytest.mark.parametrize("draft", [True, False])
def test_rows_without_a_distribution(draft):
    rng = np.random.default_rng(4)
    for value in (-np.inf, np.nan, np.inf):
        for spot in ("all", "one"):
            if spot == "one" and value == -np.inf:
                continue
            b = batch(rng, [3, 3, 3, 2, 3], 9000, False)
            b["t"] = np.array([1, 1, 0, 0, 0.5], np.float32)
            for r in (0, 4, 6, 10, 13):
                at = slice(None) if spot == "all" else 8999
                b["x"][r, at] = value
            b["tx"] = dev(b["x"].astype(np.float32))
            b["tokens"][3] = int(np.argmax(b["x"][3]))
            check(b, draft)
    if draft:
        b = batch(rng, [3, 3], 500, False)
        b["y"][0] = -np.inf
        b["y"][3, 7] = np.nan
        b["ty"] = dev(b["y"].astype(np.float32))
        check(b)


def test_tokens_outside_and_refused_ones():
    rng = np.random.default_rng(5)
    for draft in (True, False):
        b = batch(rng, [3, 3, 3, 3, 3, 3], 300, False)
        b["t"] = np.array([1, 1, 1, 0, 0, 1], np.float32)
        b["tokens"][[0, 3, 6, 9, 12]] = [-1, 300, 2 ** 31 - 1, -5, 301]
        b["tokens"][[2, 5, 8, 11, 14, 17]] = -(2 ** 31)   # the last rows' are not looked at
        b["x"][15, b["tokens"][15]] = -np.inf              # ruled out by the target
        b["tx"] = dev(b["x"].astype(np.float32))
        b["u"][15] = 0.0
        acc, _ = check(b, draft)
        assert (acc == 0).all()


def test_borders_of_the_numbers():
    rng = np.random.default_rng(6)
    b = batch(rng, [2] * 12, 400, False)
    b["u"][:] = 0.0
    assert (check(b)[0] == 1).all()
    one = np.float32(1.0) - np.float32(2.0 ** -24)
    b["un"][:] = one   # the last token with any weight
    check(b)
    b["un"][:] = 0.0   # the first
    _, nxt = check(b)
    for s in range(12):
        assert nxt[s] == int(np.nonzero(np.isfinite(b["x"][2 * s + 1]))[0][0])
    # all weight on the drafted token: nothing is left without it
    x = np.full((2, 50), -np.inf)
    x[:, 7] = 1.0
    b = dict(tx=dev(x.astype(np.float32)), ty=None, x=x, y=None, starts=np.array([0, 2], np.int32),
             tokens=np.array([7, 0], np.int32), u=np.array([1.0, 0.0], np.float32), un=np.array([0.5], np.float32), t=None)
    acc, nxt = check(b, draft=False)
    assert acc[0] == 0 and nxt[0] == 7


def test_greedy_ties_and_infinities():
    x = np.zeros((4, 20000))
    x[0, [15000, 9000, 19999]] = 5.0
    x[1, [1, 2]] = -0.0
    x[2] = -np.inf
    x[2, 12345] = -1e30
    x[3, 8192] = 3e38
    b = dict(tx=dev(x.astype(np.float32)), x=x.astype(np.float32).astype(np.float64), starts=np.array([0, 4], np.int32),
             tokens=np.array([9000, 0, 12345, 0], np.int32), u=np.ones(4, np.float32), un=np.zeros(1, np.float32),
             t=np.zeros(1, np.float32))
    b["ty"], b["y"] = b["tx"], b["x"]
    for draft in (True, False):
        acc, nxt = check(b, draft)
        assert acc[0] == 3 and nxt[0] == 8192


@pytest.mark.parametrize("bf16", [False, True])
def test_empty_sequences_strides_and_foreign_rows(bf16):
    rng = np.random.default_rng(7)
    b = batch(rng, [0, 3, 0, 0, 4, 2, 0], 1000, bf16)
    acc, nxt = check(b)
    assert nxt[0] == -1 and nxt[2] == -1 and nxt[6] == -1
    for pad in (8, 3):   # rows apart: aligned, and not
        wide = torch.full((9, 1000 + pad), 50.0, dtype=b["tx"].dtype, device=DEV)
        wide[:, :1000] = b["tx"]
        wy = torch.full((9, 1000 + pad), 50.0, dtype=b["tx"].dtype, device=DEV)
        wy[:, :1000] = b["ty"]
        check(dict(b, tx=wide[:, :1000], ty=wy[:, :1000]))
        check(dict(b, tx=wide[:, :1000]))   # unlike strides
    # rows before the first and behind the last sequence
    starts = np.array([2, 5, 8], np.int32)
    c = dict(b, starts=starts, un=b["un"][:2])
    check(c)
    for odd in ([-3, 2, 100], [9, 4, 6], [2 ** 31 - 1, -(2 ** 31), 0]):
        r = g.gguf_verify_draft(b["tx"], dev(b["tokens"]), dev(b["u"]), dev(b["un"][:2]), dev(np.array(odd, np.int32)),
                                draft=b["ty"])
        assert (host(r.accepted) >= 0).all() and (host(r.next_tokens) < 1000).all()


def test_many_rows_of_one_sequence():
    rng = np.random.default_rng(8)
    b = batch(rng, [70, 130], 600, False, noise=0.01)
    check(b)
    b = batch(rng, [70, 130], 600, False, noise=0.01, ruled_out=False)   # drafts seldom refused
    acc, _ = check(b)
    assert acc.max() > 20


def test_streams_and_a_graph():
    rng = np.random.default_rng(9)
    b = batch(rng, [5, 3, 8, 1], 20000, False)
    b["t"] = np.array([0.7, 0.0, 1.0, 1.0], np.float32)
    d = {k: dev(b[k]) for k in ("tokens", "u", "un", "starts", "t")}

    def call(**kw):
        return g.gguf_verify_draft(b["tx"], d["tokens"], d["u"], d["un"], d["starts"], draft=b["ty"], temperature=d["t"], **kw)
    want = [host(x) for x in call()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [call(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(np.array_equal(host(x), w) for o in outs for x, w in zip(o, want))
    ws = torch.full((g.gguf_verify_draft_workspace(17, 4, 20000, True),), 0xFF, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call(workspace=ws)
    for i in range(4):
        d["u"].copy_(dev(rng.random(17).astype(np.float32)))
        d["un"].copy_(dev(rng.random(4).astype(np.float32)))
        want = [host(x) for x in call()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host(x), w) for x, w in zip(r, want)), i


def test_refusals_of_the_binding():
    x = torch.zeros((4, 50), device=DEV)
    ok = dict(target=x, tokens=torch.zeros(4, dtype=torch.int32, device=DEV), uniform=torch.zeros(4, device=DEV),
              uniform_next=torch.zeros(2, device=DEV), row_start=dev(np.array([0, 2, 4], np.int32)), draft=x.clone())
    g.gguf_verify_draft(**ok)
    for bad in [dict(target=x.half()), dict(target=x[0]), dict(tokens=ok["tokens"][:3]), dict(tokens=ok["tokens"].long()),
                dict(uniform=ok["uniform"].double()), dict(uniform_next=ok["uniform"]), dict(draft=x[:3]),
                dict(draft=x.bfloat16()), dict(row_start=ok["row_start"].long()), dict(temperature=ok["uniform"]),
                dict(row_start=ok["row_start"][:0]), dict(workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))]:
        with pytest.raises(ValueError):
            g.gguf_verify_draft(**dict(ok, **bad))
