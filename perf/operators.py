"""What is measured of the serving-side operators: the paged key-value cache, the
attention of one new token over it, eviction from it, and the log probabilities
read from the output head.

Each case is one call as a serving program makes it, with the operators in plain
torch form (fp32, rounded once at the end) or, where `own` is true, through the
library. Head shapes are those of the decode workload here (16 query heads over
4 key-value heads of 128) and generic ones; the vocabulary is its 128256.

The cache's layout (both sides read the same bytes): pages of `page` slots,
K as [page][kv head][slot][dim], V transposed as [page][kv head][dim][slot];
Q8_0 keeps, per page and kv head, the int8 codes in that order and after them
the fp16 scales of 32 dims each (K [slot][dim / 32], V [dim / 32][slot]).
`weight` (fp32, accumulated attention) and `pos` (int32) are [page][kv head][slot].
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
GGUF_IDS = {"f16": 1, "bf16": 30, "q8_0": 8}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the new token of every running sequence goes into the cache (fp32 GEMV outputs)
        dict(name="append one token x 16", op="append", type="bf16", src="f32", seqs=16, tokens=1,
             kv_heads=4, dim=128, page=16, longest=4096),
        # prompts go into the cache (bf16 prefill outputs)
        dict(name="append prompts 8 x 4096", op="append", type="f16", src="bf16", seqs=8, tokens=4096,
             kv_heads=4, dim=128, page=64, longest=8192),
        # a short conversation, batch 1: latency
        dict(name="attend 1 x 300", op="attend", type="f16", seqs=1, heads=16, kv_heads=4, dim=128, page=16,
             shortest=300, longest=300, window=0, track=False),
        # one long context, batch 1: the work is split over the cache's length
        dict(name="attend 1 x 32768", op="attend", type="bf16", seqs=1, heads=16, kv_heads=4, dim=128,
             page=64, shortest=32768, longest=32768, window=0, track=False),
        # a batch of uneven sequences, empty slots among them, whose attention weights are accumulated
        dict(name="attend 64 x 0..4096 tracked", op="attend", type="bf16", seqs=64, heads=16, kv_heads=4,
             dim=128, page=32, shortest=0, longest=4096, window=0, track=True),
        # a large batch of long sequences: bandwidth
        dict(name="attend 32 x 1..16384", op="attend", type="f16", seqs=32, heads=32, kv_heads=8, dim=128,
             page=128, shortest=1, longest=16384, window=0, track=False),
        # long contexts kept in 8 bits
        dict(name="attend 8 x 32768 q8_0", op="attend", type="q8_0", seqs=8, heads=16, kv_heads=4, dim=128,
             page=64, shortest=20001, longest=32768, window=0, track=False),
        # every step at the budget: one slot per head makes room
        dict(name="evict 16 x 4097 to 4096", op="evict", type="bf16", seqs=16, kv_heads=4, dim=128, page=32,
             shortest=4097, longest=4097, budget=4096, recent=256),
        # after a prompt: most of it goes
        dict(name="evict 4 x 32768 to 8192", op="evict", type="f16", seqs=4, kv_heads=4, dim=128, page=64,
             shortest=32768, longest=32768, budget=8192, recent=1024),
        # one decode step's head output
        dict(name="logprobs 1 x 128256", op="logprobs", type="f32", rows=1, vocab=128256, given=1, top=5),
        # a small batch's head outputs
        dict(name="logprobs 64 x 128256", op="logprobs", type="f32", rows=64, vocab=128256, given=1, top=20),
        # a prompt scored
        dict(name="logprobs 1024 x 128256 bf16", op="logprobs", type="bf16", rows=1024, vocab=128256, given=4,
             top=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict", "logprobs", "logprobs"])
    if op == "logprobs":
        vocab = _log(rng, 997, 151936)
        rows = max(1, min(_log(rng, 1, 1024), 1024 * 128256 // vocab // 2))
        return dict(op=op, type=rng.choice(["f32", "bf16"]), rows=rows if vocab < 60000 else min(rows, 400),
                    vocab=vocab, given=rng.randint(1, 8), top=rng.randint(0, 32))
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 192, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        tokens = rng.choice([1, 1, _log(rng, 2, 4096)])
        seqs = rng.randint(1, 128) if tokens == 1 else rng.randint(1, 4)
        return dict(op=op, type=rng.choice(["f16", "bf16"]), src=rng.choice(["f32", "bf16"]), seqs=seqs,
                    tokens=tokens, kv_heads=kv_heads, dim=dim, page=page,
                    longest=tokens + rng.randint(0, 2000))
    seqs = rng.choice([1, rng.randint(2, 8), rng.randint(9, 64)])
    # at most what the largest listed case reads
    most = 16 * 16384 * 8 * 128 // (seqs * kv_heads * dim)
    longest = min(_log(rng, 1, 65536), most)
    if op == "attend":
        heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16])
        return dict(op=op, type=rng.choice(["f16", "bf16", "q8_0"]), seqs=seqs, heads=heads, kv_heads=kv_heads,
                    dim=dim, page=page, shortest=rng.choice([0, 1, longest]), longest=longest,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), track=rng.choice([False, False, True]))
    longest = max(2, min(longest, 32768, most // 4))
    budget = rng.choice([longest - 1, rng.randint(1, longest)])
    return dict(op=op, type=rng.choice(["f16", "bf16"]), seqs=seqs, kv_heads=kv_heads, dim=dim, page=page,
                shortest=rng.choice([1, longest]), longest=longest, budget=budget,
                recent=rng.randint(0, budget))


# ------------------------------------------------------------------ inputs

def _lengths(case, gen):
    """Lengths of the batch: spread over shortest .. longest, one of each."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    x = torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    x[0] = hi
    if n > 1:
        x[-1] = lo
    return x


def _page_table(seqs, pages, gen):
    """Pages handed out in a mixed order, a few of them to nobody."""
    n = seqs * pages
    return n + 3, torch.randperm(n + 3, generator=gen, device="cuda")[:n].to(torch.int32).view(seqs, pages)


def _cache_half(case, n_pages, gen, transposed):
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    if case["type"] != "q8_0":
        shape = (n_pages, h, d, p) if transposed else (n_pages, h, p, d)
        return torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[case["type"]])
    codes = torch.randint(-127, 128, (n_pages, h, p * d), generator=gen, device="cuda", dtype=torch.int8)
    scales = (0.01 + 0.02 * torch.rand((n_pages, h, p * d // 32), generator=gen, device="cuda")).half()
    return torch.cat([codes.view(torch.uint8), scales.view(torch.uint8)], -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "logprobs":
        n, v = case["rows"], case["vocab"]
        x = 2.0 * torch.randn((n, v), generator=gen, device="cuda")
        peaks = torch.randint(0, v // 20, (n, 20), generator=gen, device="cuda")
        peaks += v // 20 * torch.arange(20, device="cuda")
        x.scatter_(1, peaks, 12.0 * torch.rand((n, 20), generator=gen, device="cuda"))
        # tokens that the sampler has ruled out
        x[:, torch.randint(0, v, (max(1, v // 200),), generator=gen, device="cuda")] = -math.inf
        tokens = torch.randint(0, v, (n, case["given"]), generator=gen, device="cuda", dtype=torch.int32)
        tokens[:, 0] = peaks[:, 0].to(torch.int32)   # one that is likely
        st = dict(case=case, logits=x if case["type"] == "f32" else x.to(torch.bfloat16), tokens=tokens)
        if own:
            import gguf_block_quant_dequant_amd as g
            st["workspace"] = torch.empty(max(16, g.gguf_logprobs_workspace(n, v, case["top"])),
                                          dtype=torch.uint8, device="cuda")
        return st
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    pages = -(-case["longest"] // p) + (1 if op == "append" else 0)
    n_pages, table = _page_table(case["seqs"], pages, gen)
    st = dict(case=case, table=table, k=_cache_half(case, n_pages, gen, False),
              v=_cache_half(case, n_pages, gen, True))
    if op == "append":
        n, t = case["seqs"], case["tokens"]
        start = torch.randint(0, case["longest"] - t + 1, (n, 1), generator=gen, device="cuda")
        dt = torch.float32 if case["src"] == "f32" else torch.bfloat16
        st["new_k"] = torch.randn((n * t, h * d), generator=gen, device="cuda", dtype=dt)
        st["new_v"] = torch.randn((n * t, h * d), generator=gen, device="cuda", dtype=dt)
        st["slot"] = (start + torch.arange(t, device="cuda")).reshape(-1).to(torch.int32)
        st["seq"] = torch.arange(n, device="cuda", dtype=torch.int32).repeat_interleave(t)
    else:
        lengths = _lengths(case, gen)
        # weight, pos and lengths in one buffer, so that a pass can start from the same values
        m = n_pages * h * p
        small = torch.empty(2 * m + case["seqs"], dtype=torch.int32, device="cuda")
        st["weight"] = small[:m].view(torch.float32).view(n_pages, h, p)
        st["pos"], st["lengths"] = small[m:2 * m].view(n_pages, h, p), small[2 * m:]
        # accumulated weights: heavy-tailed, some slots never attended (ties)
        w = torch.exp(2.0 * torch.randn((n_pages, h, p), generator=gen, device="cuda"))
        st["weight"].copy_(w * (torch.rand((n_pages, h, p), generator=gen, device="cuda") > 0.05))
        # positions in a mixed order, as earlier evictions leave them
        n = pages * p
        order = torch.rand((case["seqs"], h, n), generator=gen, device="cuda").argsort(-1).to(torch.int32)
        st["pos"].zero_()
        st["pos"][table.long()] = order.view(case["seqs"], h, pages, p).transpose(1, 2)
        st["lengths"].copy_(lengths)
        st["small"], st["small0"] = small, small.clone()
    if op == "attend":
        st["q"] = 2.0 * torch.randn((case["seqs"], case["heads"], d), generator=gen, device="cuda")
    if own:
        import gguf_block_quant_dequant_amd as g
        st["cache"] = g.KvCache(st["k"], st["v"], GGUF_IDS[case["type"]], h, d, p, weight=st.get("weight"),
                                pos=st.get("pos"))
        if op == "attend":
            st["out"] = torch.empty_like(st["q"])
            need = g.gguf_attn_decode_workspace(st["cache"], case["seqs"], case["heads"], case["longest"],
                                                case["track"])
            st["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
        if op == "evict":
            need = g.gguf_kv_evict_workspace(st["cache"], case["seqs"], case["longest"], case["budget"])
            st["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if op == "evict":
        state["small"].copy_(state["small0"])   # both sides: weights, positions and lengths as before the call
    if own:
        return {"append": _own_append, "attend": _own_attend, "evict": _own_evict,
                "logprobs": _own_logprobs}[op](state, case)
    return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict,
            "logprobs": _plain_logprobs}[op](state, case)


def _own_append(st, case):
    import gguf_block_quant_dequant_amd as g
    g.gguf_kv_append(st["cache"], st["new_k"], st["new_v"], st["table"], st["slot"], seq=st["seq"])
    return {"k": st["k"], "v": st["v"]}


def _own_attend(st, case):
    import gguf_block_quant_dequant_amd as g
    out = g.gguf_attn_decode(st["cache"], st["q"], st["table"], st["lengths"], case["longest"],
                             window=case["window"], track=case["track"], out=st["out"],
                             workspace=st["workspace"])
    return {"out": out, "weight": st["weight"]} if case["track"] else {"out": out}


def _own_evict(st, case):
    import gguf_block_quant_dequant_amd as g
    g.gguf_kv_evict(st["cache"], st["table"], st["lengths"], case["longest"], case["budget"],
                    recent=case["recent"], workspace=st["workspace"])
    return {"k": st["k"], "v": st["v"], "weight": st["weight"], "pos": st["pos"], "lengths": st["lengths"]}


def _own_logprobs(st, case):
    import gguf_block_quant_dequant_amd as g
    r = g.gguf_logprobs(st["logits"], st["tokens"], top_k=case["top"], workspace=st["workspace"])
    return _named(r.token_logprobs, r.entropy, r.top_ids, r.top_logprobs, case)


def _named(lp, entropy, ids, top, case):
    got = {"token_logprobs": lp, "entropy": entropy}
    if case["top"]:
        got["top_ids"], got["top_logprobs"] = ids, top
    return got


def _plain_append(st, case):
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    seq, slot = st["seq"].long(), st["slot"].long()
    page, at = st["table"][seq, slot // p].long(), slot % p
    st["k"][page, :, at] = st["new_k"].float().view(-1, h, d).to(st["k"].dtype)
    st["v"][page, :, :, at] = st["new_v"].float().view(-1, h, d).to(st["v"].dtype)
    return {"k": st["k"], "v": st["v"]}


def _plain_values(x, table, case, transposed):
    """The cache's fp32 values by sequence: [seqs, kv heads, positions, dim]."""
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    x = x[table.long()]
    shape = x.shape[:3] + ((d, p) if transposed else (p, d))
    if case["type"] == "q8_0":
        codes = x[..., :p * d].view(torch.int8).float().view(shape)
        scales = x[..., p * d:].contiguous().view(torch.float16).float()
        if transposed:
            x = codes.view(*x.shape[:3], d // 32, 32, p) * scales.view(*x.shape[:3], d // 32, 1, p)
        else:
            x = codes.view(*x.shape[:3], p, d // 32, 32) * scales.view(*x.shape[:3], p, d // 32, 1)
        x = x.view(shape)
    x = x.float()
    if transposed:
        x = x.transpose(-1, -2)
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], h, -1, d)


def _plain_attend(st, case):
    s, h, d, p = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    k = _plain_values(st["k"], st["table"], case, False)
    n = k.shape[2]
    q = st["q"].view(s, h, -1, d) * (1.0 / math.sqrt(d))
    scores = torch.matmul(q, k.transpose(-1, -2))
    at, lengths = torch.arange(n, device="cuda"), st["lengths"].view(s, 1, 1, 1)
    seen = at < lengths
    if case["window"]:
        seen = seen & (at >= lengths - case["window"])
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(scores - top), 0.0)
    total = e.sum(-1, keepdim=True)
    e = torch.where(total > 0, e / total, 0.0)
    v = _plain_values(st["v"], st["table"], case, True)
    v = torch.where(seen.view(s, 1, n, 1), v, 0.0)
    out = torch.matmul(e, v).view(s, case["heads"], d)
    if not case["track"]:
        return {"out": out}
    w = e.sum(2).view(s, h, -1, p).transpose(1, 2)
    st["weight"][st["table"].long()] += w
    return {"out": out, "weight": st["weight"]}


def _plain_evict(st, case):
    s, h, p, b = case["seqs"], case["kv_heads"], case["page"], case["budget"]
    table = st["table"].long()
    n = table.shape[1] * p
    weight = st["weight"][table].transpose(1, 2).reshape(s, h, n)
    pos = st["pos"][table].transpose(1, 2).reshape(s, h, n)
    at, lengths = torch.arange(n, device="cuda"), st["lengths"].long().view(s, 1, 1)
    valid = (at < lengths).expand(s, h, n)
    newest = torch.where(valid, pos, -1).amax(-1, keepdim=True)
    key = torch.where(valid & (pos > newest - case["recent"]), math.inf, weight)
    key = torch.where(valid, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(valid).scatter(-1, order[..., :b], True) & valid
    hole = ~keep & (at < b) & (lengths > b)
    tail = keep & (at >= b)
    tails = torch.sort((~tail).to(torch.int8), dim=-1, stable=True).indices
    filler = torch.gather(tails, -1, (torch.cumsum(hole.to(torch.int32), -1) - 1).clamp(min=0).long())
    src = torch.where(hole, filler, at)[..., :b]
    dst = at[:b].expand_as(src)
    row, head = torch.arange(s, device="cuda").view(s, 1, 1), torch.arange(h, device="cuda").view(1, h, 1)
    sp, so, dp, do = table[row, src // p], src % p, table[row, dst // p], dst % p
    moved = [x[sp, head, so] for x in (st["k"], st["weight"], st["pos"])]
    moved_v = st["v"][sp, head, :, so]
    for x, m in zip((st["k"], st["weight"], st["pos"]), moved):
        x[dp, head, do] = m
    st["v"][dp, head, :, do] = moved_v
    st["lengths"].clamp_(max=b)
    return {"k": st["k"], "v": st["v"], "weight": st["weight"], "pos": st["pos"], "lengths": st["lengths"]}


def _plain_logprobs(st, case):
    x = st["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    tokens = st["tokens"].long()
    lp = torch.gather(x, 1, tokens) - lse
    p = e / total
    entropy = -torch.where(p > 0, p * (x - lse), 0.0).sum(-1)
    if not case["top"]:
        return _named(lp, entropy, None, None, case)
    order = torch.sort(x, dim=-1, descending=True, stable=True)
    ids = order.indices[:, :case["top"]].to(torch.int32)
    return _named(lp, entropy, ids, order.values[:, :case["top"]] - lse, case)


# ------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    if op == "logprobs":
        n, v = case["rows"], case["vocab"]
        return {"bytes": n * v * (4 if case["type"] == "f32" else 2) + n * (8 * case["given"] + 8 * case["top"] + 4),
                "flops": 6.0 * n * v}
    h, d = case["kv_heads"], case["dim"]
    slot = 2 * h * d * (34 / 32 if case["type"] == "q8_0" else 2)   # K and V of one position
    if op == "append":
        t = case["seqs"] * case["tokens"]
        return {"bytes": t * (slot + 2 * h * d * (4 if case["src"] == "f32" else 2) + 8), "flops": 2.0 * t * h * d}
    seen = case["seqs"] * (case["shortest"] + case["longest"]) / 2
    if op == "attend":
        if case["window"]:
            seen = min(seen, case["seqs"] * case["window"])
        return {"bytes": seen * (slot + (8 * h if case["track"] else 0)) + 8 * case["seqs"] * case["heads"] * d,
                "flops": 4.0 * seen * case["heads"] * d}
    # eviction: weights and positions read; a kept slot behind the budget moves into a hole
    out = max(0.0, seen / case["seqs"] - case["budget"])
    moves = case["seqs"] * out * case["budget"] / max(seen / case["seqs"], 1)
    return {"bytes": seen * 8 * h + moves * 2 * (slot + 8 * h), "flops": 4.0 * seen * h}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict,
            "logprobs": _exact_logprobs}[case["op"]](st, case)


def _exact_append(st, case):
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    got = {"k": st["k"].double(), "v": st["v"].double()}
    if case["tokens"] == 1:
        table = st["table"].tolist()
        for t, (s, i) in enumerate(zip(st["seq"].tolist(), st["slot"].tolist())):
            pg = table[s][i // p]
            got["k"][pg, :, i % p, :] = st["new_k"][t].double().view(h, d)
            got["v"][pg, :, :, i % p] = st["new_v"][t].double().view(h, d)
        return got
    for s in range(case["seqs"]):   # one sequence: its positions in order, page by page
        t0, first = s * case["tokens"], int(st["slot"][s * case["tokens"]])
        done = 0
        while done < case["tokens"]:
            i = first + done
            n = min(p - i % p, case["tokens"] - done)
            pg = int(st["table"][s, i // p])
            for name, new in (("k", st["new_k"]), ("v", st["new_v"])):
                rows = new[t0 + done:t0 + done + n].double().view(n, h, d)
                if name == "k":
                    got["k"][pg, :, i % p:i % p + n, :] = rows.permute(1, 0, 2)
                else:
                    got["v"][pg, :, :, i % p:i % p + n] = rows.permute(1, 2, 0)
            done += n
    return got


def _exact_kv(st, case, s, n):
    """K and V of the first n positions of one sequence: fp64 [kv heads, n, dim]."""
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    pages = st["table"][s, :-(-n // p)].long()
    k, v = st["k"][pages], st["v"][pages]
    if case["type"] == "q8_0":
        def scales(x):
            return x[:, :, p * d:].contiguous().view(torch.float16).double()

        def codes(x):
            return x[:, :, :p * d].contiguous().view(torch.int8).double()
        k = codes(k).view(-1, h, p, d) * scales(k).view(-1, h, p, d // 32).repeat_interleave(32, 3)
        v = codes(v).view(-1, h, d, p) * scales(v).view(-1, h, d // 32, p).repeat_interleave(32, 2)
    k = k.double().transpose(0, 1).reshape(h, -1, d)[:, :n]
    v = v.double().permute(1, 0, 3, 2).reshape(h, -1, d)[:, :n]
    return k, v


def _exact_attend(st, case):
    h, d, p = case["kv_heads"], case["dim"], case["page"]
    group = case["heads"] // h
    out = torch.zeros((case["seqs"], case["heads"], d), dtype=torch.float64, device="cuda")
    weight = st["weight"].double() if case["track"] else None
    for s, n in enumerate(st["lengths"].tolist()):
        if n <= 0:
            continue
        first = max(0, n - case["window"]) if case["window"] else 0
        k, v = _exact_kv(st, case, s, n)
        k, v = k[:, first:], v[:, first:]
        for j in range(h):
            q = st["q"][s, j * group:(j + 1) * group].double()
            a = torch.softmax(q @ k[j].T.contiguous() / math.sqrt(d), -1)
            out[s, j * group:(j + 1) * group] = a @ v[j]
            if case["track"]:
                full = torch.zeros(-(-n // p) * p, dtype=torch.float64, device="cuda")
                full[first:n] = a.sum(0)
                weight[st["table"][s, :-(-n // p)].long(), j] += full.view(-1, p)
    return {"out": out, "weight": weight} if case["track"] else {"out": out}


def _exact_evict(st, case):
    import numpy as np
    h, p, b = case["kv_heads"], case["page"], case["budget"]
    got = {"k": st["k"].double(), "v": st["v"].double(), "weight": st["weight"].double(),
           "pos": st["pos"].clone(), "lengths": st["lengths"].clamp(max=b)}
    table = st["table"].cpu().numpy()
    weight, pos = st["weight"].cpu().numpy(), st["pos"].cpu().numpy()
    for s, n in enumerate(st["lengths"].tolist()):
        if n <= b:
            continue
        at = np.arange(n)
        pages, slots = table[s][at // p], at % p
        for j in range(h):
            w, q = weight[pages, j, slots].astype(np.float64), pos[pages, j, slots]
            w[q > int(q.max()) - case["recent"]] = np.inf
            kept = np.sort(np.lexsort((at, -w))[:b])
            src = kept[kept >= b]
            dst = np.setdiff1d(np.arange(b), kept)
            if not len(src):
                continue
            sp, so, dp, do = (torch.from_numpy(x.astype(np.int64)).cuda()
                              for x in (pages[src], slots[src], pages[dst], slots[dst]))
            for name in ("k", "weight", "pos"):
                got[name][dp, j, do] = got[name][sp, j, so].clone()
            got["v"][dp, j, :, do] = got["v"][sp, j, :, so].clone()
    return got


def _exact_logprobs(st, case):
    n, k = case["rows"], case["top"]
    lps, ents, ids, tops = [], [], [], []
    for r in range(0, n, 64):
        x = st["logits"][r:r + 64].double()
        lse = torch.logsumexp(x, -1, keepdim=True)
        lps.append(torch.gather(x, 1, st["tokens"][r:r + 64].long()) - lse)
        lp = x - lse
        ents.append(-(lp.exp() * torch.where(torch.isinf(lp), 0.0, lp)).sum(-1))
        at = torch.arange(x.shape[1], device="cuda").expand_as(x)
        got_i, got_v = [], []
        for _ in range(k):
            best = x.amax(-1, keepdim=True)
            i = torch.where(x == best, at, x.shape[1]).amin(-1, keepdim=True)
            got_i.append(i)
            got_v.append(best - lse)
            x = x.scatter(1, i, -math.inf)
        if k:
            ids.append(torch.cat(got_i, 1).to(torch.int32))
            tops.append(torch.cat(got_v, 1))
    return _named(torch.cat(lps), torch.cat(ents), torch.cat(ids) if k else None,
                  torch.cat(tops) if k else None, case)
