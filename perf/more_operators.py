"""Cases of what closes one speculative-verify step and opens the next, and of the 4-bit cache in between, with their
plain forms.

* attn4: attention of each request's new tokens over a paged cache held in NVFP4 (E2M1 codes, an E4M3 scale per 16)
* append4: rotary positions of q and k, the append of k and v to such a cache, and the values that it then stands for
* drafts: which drafted tokens a verify pass accepts, from the target's logits or probabilities and given random
  numbers, and the token that follows them
* tables: the next step's token offsets, lengths, page table and slots from what was accepted, on the GPU

A batch is `requests` requests; request r brings n_r new tokens (`mix`: all `new`, or spread) and has kv_r tokens in the
cache when these are in it.  Both follow from the case alone, so that work() counts exactly what is read.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the smallest call: one short request, one token
        dict(name="attn4_one", op="attn4", requests=1, new=1, kv=257, mix="even", heads=16, kv_heads=4, dim=128,
             page=16, window=0, sinks=0),
        # the verify pass of 16 requests x (1 + 12 drafts) over uneven contexts
        dict(name="attn4_verify", op="attn4", requests=16, new=13, kv=4096, mix="contexts", heads=32, kv_heads=8,
             dim=128, page=64, window=0, sinks=0),
        # long contexts, one token each: the cache is all there is to read
        dict(name="attn4_long", op="attn4", requests=4, new=1, kv=131072, mix="contexts", heads=32, kv_heads=8,
             dim=128, page=64, window=0, sinks=0),
        # chunks of two prompts after earlier chunks: matrix-core work
        dict(name="attn4_chunk", op="attn4", requests=2, new=2048, kv=10007, mix="ragged", heads=32, kv_heads=8,
             dim=128, page=64, window=0, sinks=0),
        # the verify pass's tokens into the cache, positions scaled for a longer context
        dict(name="append4_verify", op="append4", requests=16, new=13, kv=2000, mix="even", heads=32, kv_heads=8,
             dim=128, rot=128, page=64, interleaved=False, scaling="yarn", offset=0),
        # prompts of uneven lengths, half of each head rotated, interleaved pairs, positions far from zero
        dict(name="append4_prompt", op="append4", requests=4, new=2048, kv=2500, mix="ragged", heads=32, kv_heads=8,
             dim=128, rot=64, page=64, interleaved=True, scaling="linear", offset=1000003),
        # one request with four drafts of a small draft model: latency
        dict(name="drafts_one", op="drafts", requests=1, new=5, mix="even", vocab=32000, given="logits", bits=16,
             temperature=1.0, draft="probs", cut=0.0),
        # the verify pass of 16 requests x (1 + 12 drafts): all logits are read once
        dict(name="drafts_verify", op="drafts", requests=16, new=13, mix="even", vocab=131072, given="logits", bits=16,
             temperature=0.8, draft="probs", cut=0.0),
        # a large batch of greedy requests whose drafts were looked up, not drawn
        dict(name="drafts_greedy", op="drafts", requests=64, new=13, mix="ragged", vocab=128000, given="logits",
             bits=16, temperature=0.0, draft="none", cut=0.0),
        # the program filtered and normalized the probabilities itself; a vocabulary of odd size
        dict(name="drafts_probs", op="drafts", requests=64, new=9, mix="ragged", vocab=50001, given="probs", bits=32,
             temperature=1.0, draft="probs", cut=6.0),
        # the step after a verify pass of 16 requests
        dict(name="tables_verify", op="tables", requests=16, new=13, kv=4096, page=64, prompts=0),
        # a large server's step: most requests decode, every sixteenth starts on a prompt, some have ended
        dict(name="tables_server", op="tables", requests=2048, new=5, kv=16384, page=16, prompts=4096),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn4", "attn4", "append4", "drafts", "drafts", "tables"])
    if op == "drafts":
        requests, given = _spread(rng, 1, 128), rng.choice(["logits", "logits", "probs"])
        new = _spread(rng, 1, 16)
        vocab = min(_spread(rng, 1000, 262144), (1 << 26) // (requests * new))
        draft = rng.choice(["probs", "probs", "none"])
        return dict(op=op, requests=requests, new=new, mix=rng.choice(["even", "ragged"]), vocab=vocab, given=given,
                    bits=rng.choice([16, 32]) if given == "logits" else 32,
                    temperature=rng.choice([0.0, 0.7, 1.0, 1.3]) if given == "logits" else 1.0, draft=draft,
                    cut=rng.choice([0.0, 5.0]))
    if op == "tables":
        page, requests = rng.choice([16, 32, 64, 128]), _spread(rng, 1, 4096)
        kv = min(_spread(rng, 64, 131072), (1 << 22) * page // requests)
        return dict(op=op, requests=requests, new=_spread(rng, 1, 16), kv=kv, page=page,
                    prompts=rng.choice([0, min(kv // 2, _spread(rng, 16, 4096))]))
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    requests, mix = _spread(rng, 1, 64), rng.choice(["even", "contexts", "ragged"])
    new = rng.choice([1, _spread(rng, 2, 16), _spread(rng, 16, 2048)])
    if op == "append4":
        new = min(new, max(1, (1 << 25) // (requests * (heads + 2 * kv_heads) * dim)))
        kv = new + min(_spread(rng, 1, 4096), max(1, (1 << 24) // (requests * kv_heads * dim)))
        return dict(op=op, requests=requests, new=new, kv=kv, mix=mix, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), page=page, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), offset=rng.choice([0, 0, 70001, 1000003]))
    # no more cache, scores or products than the listed cases have
    new = min(new, max(1, (1 << 24) // (requests * heads)))
    most = min((1 << 29) // (requests * kv_heads * dim), (1 << 30) // (requests * heads * new),
               (1 << 37) // (requests * heads * new * dim))
    kv = new + min(_spread(rng, 1, 131072), max(1, most - new))
    window = rng.choice([0, 0, _spread(rng, 16, 4096)])
    return dict(op=op, requests=requests, new=new, kv=kv, mix=mix, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                window=window, sinks=rng.choice([0, 1, 4, 17]) if window else 0)


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request."""
    n, kv, requests, mix = case["new"], case.get("kv", 0), case["requests"], case["mix"]
    news = [n if mix != "ragged" or r == 0 else max(1, n - (r * n * 29 // 64) % n) for r in range(requests)]
    kvs = [kv if mix == "even" or r == 0 else max(news[r], kv - (r * kv * 37 // 100) % (kv // 2 + 1))
           for r in range(requests)]
    return news, kvs


def _step(case):
    """What each request of a tables case has in the cache, brought to the step before, and brings to the next one
    (-1: it has ended)."""
    rs = range(case["requests"])
    kvs = [max(case["new"], case["kv"] - (r * case["kv"] * 37 // 100) % (case["kv"] // 2 + 1)) for r in rs]
    olds = [case["new"] if r % 5 else 1 for r in rs]
    nexts = [-1 if r % 23 == 22 else 1 if r % 3 == 2 else case["new"] for r in rs]
    if case["prompts"]:
        for r in rs[::16]:
            kvs[r], olds[r], nexts[r] = 0, 0, max(1, case["prompts"] - (r * 31) % case["prompts"])
    return kvs, olds, nexts


# ---------------------------------------------------------------- inputs

def _frequencies(case):
    """Rotary frequencies (float64 [rot / 2]) and the multiplier of cos and sin, from their published formulas:
    positions divided by a factor, a stretched base, or YaRN's blend of both by wavelength."""
    rot, base, factor, context = case["rot"], 10000.0, 8.0, 4096.0
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    j = torch.arange(rot // 2, dtype=torch.float64)
    inv = base ** (-2.0 * j / rot)
    if case["scaling"] == "linear":
        return inv / factor, 1.0
    if case["scaling"] != "yarn":
        return inv, 1.0
    turns = lambda t: rot * math.log(context / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(0, math.floor(turns(32.0))), min(rot - 1, math.ceil(turns(1.0)))
    keep = 1 - ((j - low) / max(1e-3, high - low)).clamp(0, 1)
    return inv * keep + inv / factor * (1 - keep), float(torch.tensor(0.1 * math.log(factor) + 1, dtype=torch.float32))


def _quantized(x):
    """NVFP4 of fp32 rows: packed E2M1 codes [..., n / 2] (the even element in the low half) and E4M3 scales
    [..., n / 16], the scale E4M3(max / 6), each code the E2M1 value nearest to the quotient, ties to even."""
    b = x.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1) / 6).clamp(max=448).to(E4M3)
    s = scale.float()[..., None]
    q = torch.where(s > 0, b / s, torch.zeros_like(b))
    a = q.abs()
    code = (a > 0.25).to(torch.uint8)
    for edge, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if tie_up else (a > edge)
    code = (code + 8 * torch.signbit(q).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scale, dtype):
    """The values that codes and scales stand for, [..., head size]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    table = torch.cat([table, -table])
    pair = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)        # of a byte
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (v * scale.view(E4M3).float()[..., None]).flatten(-2).to(dtype)


def _filled(pages, case, gen):
    """A cache's pool [pages, kv_heads, page, dim / 2] with what earlier steps left in it, and its scales."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    part = max(1, (1 << 27) // math.prod(shape[1:]))
    got = [_quantized(torch.randn((min(part, pages - at),) + shape[1:], device=DEV, generator=gen))
           for at in range(0, pages, part)]
    return torch.cat([g[0] for g in got]), torch.cat([g[1].view(torch.uint8) for g in got]).view(E4M3)


def _batch(case, gen):
    news, kvs = _lengths(case)
    page, requests = case.get("page", 16), case["requests"]
    most = max(1, max(-(-kv // page) for kv in kvs))
    pages = requests * most
    start = [0]
    for n in news:
        start.append(start[-1] + n)
    table = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32).reshape(requests, most)
    return dict(start=torch.tensor(start, dtype=torch.int32, device=DEV),
                kv=torch.tensor(kvs, dtype=torch.int32, device=DEV), table=table, max_new=max(news), max_kv=max(kvs),
                tokens=start[-1], pages=pages)


def _drafts(case, s, gen):
    """Logits as a model's head writes them, a draft model's that are near, and drafts from those."""
    b, vocab, requests = s["batch"], case["vocab"], case["requests"]
    tokens = b["tokens"]
    dtype = torch.bfloat16 if case["bits"] == 16 else torch.float32
    logits = torch.randn((tokens, vocab), device=DEV, generator=gen) * 3
    last = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    last[b["start"][1:].long() - 1] = True
    rows = torch.nonzero(~last)[:, 0]                     # the rows after which a draft follows
    near = logits[rows] + torch.randn((len(rows), vocab), device=DEV, generator=gen) * 0.5
    if case["cut"]:                                       # unlikely tokens that the program has ruled out
        logits.masked_fill_(logits < logits.amax(-1, keepdim=True) - case["cut"], -math.inf)
    ids = torch.randint(0, vocab, (tokens,), device=DEV, generator=gen)
    if case["draft"] == "probs":
        s["draft"] = torch.softmax(near, -1)
        noise = torch.rand(near.shape, device=DEV, generator=gen).clamp(min=1e-30).log().neg()
        ids[rows + 1] = (s["draft"] / noise).argmax(-1)   # drawn from the draft's own probabilities
    else:
        s["draft"] = None
        ids[rows + 1] = near.argmax(-1)
    s["target"] = logits.to(dtype) if case["given"] == "logits" else torch.softmax(logits, -1)
    s["ids"] = ids.to(torch.int32)
    s["temperature"] = torch.full((requests,), case["temperature"], device=DEV)
    s["u_accept"] = torch.rand(tokens, device=DEV, generator=gen)
    s["u_next"] = torch.rand(requests, device=DEV, generator=gen)


def _tables(case, s, gen):
    """The state that a server keeps between steps: lengths, pages held, the page table and a ring of free pages."""
    kvs, olds, nexts = _step(case)
    page, requests = case["page"], case["requests"]
    held = [-(-kv // page) for kv in kvs]
    # room for every request's largest length, and free pages for all
    most = max(max(held), max(-(-(kv + max(0, n)) // page) for kv, n in zip(kvs, nexts)))
    free = sum(max(0, -(-(kv + max(0, n)) // page) - h) for kv, n, h in zip(kvs, nexts, held)) + requests
    pages = sum(held) + free
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    held = ints(held)
    at = torch.arange(most, device=DEV)[None] + (held.cumsum(0) - held)[:, None]
    s["table"] = torch.where(torch.arange(most, device=DEV)[None] < held[:, None], order[at.clamp(max=pages - 1)], -1)
    taken = int(torch.randint(0, 1 << 20, (1,), device=DEV, generator=gen))
    s["ring"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    s["ring"][(taken + torch.arange(free, device=DEV)) % pages] = order[pages - free:]
    s["counts"] = torch.tensor([taken, taken + free], dtype=torch.int64, device=DEV)
    s["start"] = torch.cat([ints([0]), ints(olds).cumsum(0, dtype=torch.int32)])
    s["kv"], s["held"], s["news"] = ints(kvs), held, ints(nexts)
    s["accepted"] = (torch.rand(requests, device=DEV, generator=gen) * ints(olds)).to(torch.int32)
    s["tokens"] = sum(max(0, n) for n in nexts)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, device=DEV, generator=gen).to(torch.bfloat16)  # noqa: E731
    s = dict(case)
    if case["op"] == "tables":
        _tables(case, s, gen)
        if own:  # a server that captures its steps keeps two generations of the small arrays
            from quantized_memory_bound_amd import ocq
            s["own_before"] = ocq.PageTables(s["start"], s["kv"], s["held"], s["counts"], s["table"], s["ring"],
                                             s["page"])
            s["own_after"] = ocq.PageTables(*(torch.empty_like(s[x]) for x in ("start", "kv", "held", "counts")),
                                            s["table"], s["ring"], s["page"])
        return s
    b = s["batch"] = _batch(case, gen)
    if case["op"] == "drafts":
        _drafts(case, s, gen)
    else:
        heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
        s["k"], s["ks"] = _filled(b["pages"], case, gen)
        s["v"], s["vs"] = _filled(b["pages"], case, gen)
        if case["op"] == "append4":
            # q, k and v are what one projection wrote, side by side
            qkv = randn(b["tokens"], heads + 2 * kv_heads, dim)
            s["q"], s["new_k"], s["new_v"] = qkv.split([heads, kv_heads, kv_heads], 1)
            inv, s["multiplier"] = _frequencies(case)
            s["inv"] = inv.to(DEV)
            s["positions"] = (_positions(s) + case["offset"]).to(torch.int32) if case["offset"] else None
        else:
            s["q"] = randn(b["tokens"], heads, dim)
    if own:  # the handles that a serving program makes once: addresses and sizes of its buffers
        from quantized_memory_bound_amd import ocq
        s["own_batch"] = ocq.TokenBatch(b["start"], b["kv"], b["table"], b["max_new"], b["max_kv"])
        if case["op"] != "drafts":
            s["own_cache"] = ocq.PagedKVCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "append4":
            s["own_rope"] = ocq.Rope(s["inv"], multiplier=s["multiplier"], interleaved=case["interleaved"])
    return s


# ---------------------------------------------------------------- plain forms

def _request_of(s):
    t = torch.arange(s["batch"]["tokens"], device=DEV)
    return torch.bucketize(t, s["batch"]["start"][1:].long(), right=True), t


def _positions(s):
    """Place of every token in its request, the cached ones before it counted."""
    r, t = _request_of(s)
    b = s["batch"]
    return b["kv"].long()[r] - b["start"].long()[r + 1] + t


def _rotated(x, cos, sin, s):
    rot = s["rot"]
    y = x.double()
    if s["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _append_plain(s):
    # in 64 bits up to the fp32 values that are quantized: codes step at borders
    r, _ = _request_of(s)
    place = _positions(s)
    angle = (place if s["positions"] is None else s["positions"]).double()[:, None] * s["inv"]
    cos, sin = ((f(angle) * s["multiplier"])[:, None] for f in (torch.cos, torch.sin))
    q = _rotated(s["q"], cos, sin, s).to(torch.bfloat16)
    page, row = s["batch"]["table"][r, place // s["page"]].long(), place % s["page"]
    for x, new in (("k", _rotated(s["new_k"], cos, sin, s).float()), ("v", s["new_v"].float())):
        codes, scale = _quantized(new)
        s[x][page, :, row] = codes
        s[x + "s"].view(torch.uint8)[page, :, row] = scale.view(torch.uint8)
    return dict(q=q, k=_values(s["k"], s["ks"], torch.bfloat16), v=_values(s["v"], s["vs"], torch.bfloat16))


def _attn_plain(s):
    b, heads, kv_heads, dim = s["batch"], s["heads"], s["kv_heads"], s["dim"]
    group, requests, n = heads // kv_heads, s["requests"], b["max_new"]
    # [requests, kv_heads, tokens, dim] in 32 bits out of the pages
    k, v = (_values(s[x][b["table"].long()], s[x + "s"].view(torch.uint8)[b["table"].long()], torch.float32)
            .transpose(1, 2).flatten(2, 3) for x in ("k", "v"))
    start, kv = b["start"].long(), b["kv"].long()
    i = torch.arange(n, device=DEV)
    at = (start[:-1, None] + i).clamp(max=b["tokens"] - 1)
    q = s["q"].float()[at].reshape(requests, n, kv_heads, group, dim).transpose(1, 2).flatten(2, 3)
    score = torch.matmul(q, k.transpose(2, 3)) * dim ** -0.5
    place = kv[:, None] - (start[1:] - start[:-1])[:, None] + i
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j <= place[..., None]) & (j < kv[:, None, None])
    if s["window"]:
        seen = seen & ((j > place[..., None] - s["window"]) | (j < s["sinks"]))
    score = score.unflatten(2, (n, group)).masked_fill(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    del score
    total = p.sum(-1)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (n, group))
    out = torch.where(total[..., None] > 0, out / total[..., None], torch.zeros_like(out))
    lse = top[..., 0] + torch.log(total)
    r, t = _request_of(s)
    return dict(out=out[r, :, t - start[r]].flatten(1, 2).to(torch.bfloat16), lse=lse[r, :, t - start[r]].flatten(1, 2))


def _drafts_plain(s):
    # in 64 bits: an acceptance, and the place that a random number falls on, hang on values next to a border
    start, requests, tokens, vocab = s["batch"]["start"].long(), s["requests"], s["batch"]["tokens"], s["vocab"]
    r, t = _request_of(s)
    x = s["target"].double()
    if s["given"] == "logits":
        top = x.amax(-1, keepdim=True)
        temp = s["temperature"].double()[r][:, None]
        e = torch.exp((x - top) * (1 / temp.clamp(min=1e-30)))
        p = e / e.sum(-1, keepdim=True)
        first = torch.zeros_like(p).scatter_(1, x.argmax(-1, keepdim=True), 1.0)
        p = torch.where(temp > 0, p, first)                # temperature 0: the first of the largest
        del e, first
    else:
        p = x
    # drafts: row t is followed by token ids[t + 1], unless it is its request's last
    follows = t + 1 < start[r + 1]
    ids = s["ids"].long()[(t + 1).clamp(max=tokens - 1)]
    at = (t - r).clamp(max=max(0, tokens - requests - 1))  # row of the draft's probabilities
    px = p.gather(1, ids[:, None])[:, 0]
    qx = s["draft"].double()[at, ids] if s["draft"] is not None and tokens > requests else torch.ones_like(px)
    bad = follows & ~(s["u_accept"].double() * qx < px)
    count = (start[1:] - start[:-1] - 1).scatter_reduce(0, r, torch.where(bad, t - start[r], vocab + tokens), "amin")
    # the row that the next token comes from, and its weights
    row = start[:-1] + count
    all_in = row + 1 == start[1:]
    w = p[row]
    if s["draft"] is not None:
        if tokens > requests:
            less = (w - s["draft"].double()[at[row]]).clamp(min=0)
            w = torch.where((all_in | ~(less.sum(-1) > 0))[:, None], w, less)
    else:
        less = w.scatter(1, ids[row][:, None], 0.0)
        w = torch.where((all_in | ~(less.sum(-1) > 0))[:, None], w, less)
    c = w.cumsum(-1)
    past = (c > s["u_next"].double()[:, None] * c[:, -1:]).int()
    nxt = torch.where(past.any(-1), past.argmax(-1), vocab - 1 - (w > 0).int().flip(-1).argmax(-1))
    i = t - start[r]
    out = torch.where(i < count[r], ids, torch.where(i == count[r], nxt[r], -1))
    return dict(accepted=count.to(torch.int32), out=out.to(torch.int32))


def _tables_plain(s):
    requests, page, ring, table = s["requests"], s["page"], s["ring"], s["table"]
    most, size, tokens = table.shape[1], ring.shape[0], s["tokens"]
    old = (s["start"][1:] - s["start"][:-1]).long()
    kept = s["kv"].long() - old + torch.minimum(s["accepted"].long() + 1, old)
    ended, new = s["news"] < 0, s["news"].long().clamp(min=0)
    kept = torch.where(ended, 0, kept)
    kv, held = kept + new, s["held"].long()
    need = -(-kv // page)
    taken, given = s["counts"][0], s["counts"][1]
    want, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    want_at, back_at = want.cumsum(0) - want, back.cumsum(0) - back
    got = torch.minimum(want, (given - taken - want_at).clamp(min=0)).clamp(max=most)
    j = torch.arange(most, device=DEV)[None]
    take = (j >= held[:, None]) & (j < need[:, None])
    there = j < (held + got)[:, None]
    fresh = ring[(taken + want_at[:, None] + j - held[:, None]) % size]
    give = (j >= need[:, None]) & (j < held[:, None])
    put = torch.where(give, (given + back_at[:, None] + j - need[:, None]) % size, size)
    wide = torch.cat([ring, ring[:1]]).scatter_(0, put.flatten(), table.flatten())
    ring.copy_(wide[:-1])
    table.copy_(torch.where(take, torch.where(there, fresh, -1), table))
    start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(tokens, device=DEV)
    r = torch.bucketize(t, start[1:], right=True).clamp(max=requests - 1)
    inside = t < start[-1]
    place = kept[r] + t - start[r]
    at = table[r, (place // page).clamp(max=most - 1)].long()
    slots = torch.where(inside & (place // page < most) & (at >= 0), at * page + place % page, -1)
    got_all = torch.minimum(want.sum(), given - taken)
    ints = lambda v: v.to(torch.int32)  # noqa: E731
    return dict(start=ints(start), kv=ints(kv), held=ints(torch.minimum(need, held + got)),
                counts=torch.stack([taken + got_all, given + back.sum()]), table=table, ring=ring, slots=slots,
                positions=ints(torch.where(inside, place, -1)), requests=ints(torch.where(inside, r, -1)),
                short=ints((want.sum() - got_all)[None]))


def _run_own(s):
    from quantized_memory_bound_amd import ocq
    if s["op"] == "tables":
        after = s["own_after"]
        slots, positions, requests, short = ocq.step_tables(s["own_before"], s["news"], s["tokens"],
                                                            accepted=s["accepted"], out=after)
        return dict(start=after.q_start, kv=after.kv_lens, held=after.held, counts=after.counts,
                    table=after.page_table, ring=after.ring, slots=slots, positions=positions, requests=requests,
                    short=short)
    if s["op"] == "drafts":
        accepted, out = ocq.verify_drafts(s["target"], s["ids"], s["own_batch"], s["u_accept"], s["u_next"],
                                          draft_probs=s["draft"], temperature=s["temperature"],
                                          probabilities=s["given"] == "probs")
        return dict(accepted=accepted, out=out)
    if s["op"] == "append4":
        q = ocq.rope_append(s["q"], s["new_k"], s["new_v"], s["own_rope"], s["own_cache"], s["own_batch"],
                            positions=s["positions"])
        k, v = ocq.cache_values(s["own_cache"])
        return dict(q=q, k=k, v=v)
    out, lse = ocq.paged_attention(s["q"], s["own_cache"], s["own_batch"], window=s["window"], sinks=s["sinks"],
                                   want_lse=True)
    return dict(out=out, lse=lse)


def run(s):
    if own:
        return _run_own(s)
    return {"attn4": _attn_plain, "append4": _append_plain, "drafts": _drafts_plain, "tables": _tables_plain}[s["op"]](s)


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "tables":
        kvs, olds, nexts = _step(case)
        tokens = sum(max(0, n) for n in nexts)
        pages = sum(abs(-(-(kv + max(0, n)) // case["page"]) - -(-kv // case["page"])) if n >= 0
                    else -(-kv // case["page"]) for kv, n in zip(kvs, nexts))
        # the small arrays in and out, moved pages read and written, a slot, a position and a request a token
        return dict(bytes=case["requests"] * 32 + 8 * pages + 16 * tokens + 40, flops=8 * case["requests"])
    news, kvs = _lengths(case)
    tokens = sum(news)
    if case["op"] == "drafts":
        vocab, requests, size = case["vocab"], case["requests"], case["bits"] // 8
        drawn = requests * vocab * 4 if case["draft"] == "probs" else 0   # one row of the draft's a request
        rows = tokens if case["given"] == "logits" else requests          # given ones: the row that is drawn from
        return dict(bytes=rows * vocab * size + drawn + 12 * tokens + 12 * requests, flops=3 * rows * vocab)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    row = kv_heads * (dim // 2 + dim // 16)                               # cached bytes of one token's k (or v)
    if case["op"] == "append4":
        # the values are read out of the whole pool, in bf16
        held = case["requests"] * max(-(-kv // case["page"]) for kv in kvs) * case["page"]
        return dict(bytes=tokens * (2 * (heads + 2 * kv_heads) * dim + 2 * heads * dim + 2 * row)
                    + 2 * held * (row + 2 * kv_heads * dim), flops=3 * tokens * (heads + kv_heads) * case["rot"])
    window, sinks, read, pairs = case["window"], case["sinks"], 0, 0
    for n, kv in zip(news, kvs):
        first = kv - n                                                    # place of the first new token
        low = max(0, first - window + 1) if window else 0
        read += kv - low + min(sinks if window else 0, low)               # tokens that some row sees
        if window:
            pairs += sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(first, kv))
        else:
            pairs += n * first + n * (n + 1) // 2
    return dict(bytes=2 * row * read + tokens * heads * (4 * dim + 4) + 4 * (read // case["page"]),
                flops=4 * dim * heads * pairs)


# ---------------------------------------------------------------- in 64 bits

def _decoded(s, x, ids, head):
    """The rows of pages `ids` of one head in 64 bits: sign, exponent and mantissa of each code, times its scale."""
    byte = s[x][ids, head].reshape(-1, s["dim"] // 2)
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(1).long()
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e.double() - 1), m / 2) * (1 - 2 * (code >> 3)).double()
    scale = s[x + "s"][ids, head].reshape(-1, s["dim"] // 16).double()
    return v * scale.repeat_interleave(16, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None                                       # whole numbers throughout
    news, kvs = _lengths(case)
    if case["op"] == "drafts":
        return _drafts_exact(s, news)
    table, page = s["batch"]["table"].long().cpu(), case["page"]
    if case["op"] == "append4":
        return _append_exact(s, news, kvs, table, page)
    outs, lses, at = [], [], 0
    group = case["heads"] // case["kv_heads"]
    for r, (n, kv) in enumerate(zip(news, kvs)):
        ids = table[r, : -(-kv // page)].to(DEV)
        p = torch.arange(kv - n, kv, device=DEV)[:, None]
        j = torch.arange(kv, device=DEV)[None]
        hidden = j > p
        if case["window"]:
            hidden = hidden | ((p - j >= case["window"]) & (j >= case["sinks"]))
        for h in range(case["kv_heads"]):
            k, v = (_decoded(s, x, ids, h)[:kv] for x in ("k", "v"))
            q = s["q"][at: at + n, h * group: (h + 1) * group].double().reshape(n * group, -1)
            z = (q @ k.T / math.sqrt(case["dim"])).view(n, group, kv)
            z.masked_fill_(hidden[:, None], -math.inf)
            lse = torch.logsumexp(z, 2, keepdim=True)
            w = z.sub_(lse).exp_().view(n * group, kv)
            outs.append((w @ v).view(n, group, -1))
            lses.append(lse[..., 0])
        at += n
    # from requests x kv heads back to [tokens, heads]
    join = lambda xs: torch.cat([torch.cat(xs[i: i + case["kv_heads"]], 1)  # noqa: E731
                                 for i in range(0, len(xs), case["kv_heads"])], 0)
    return dict(out=join(outs), lse=join(lses))


def _append_exact(s, news, kvs, table, page):
    rot, at = s["rot"], 0

    def turn(x, where):  # pairs as complex numbers, turned by e^(i angle)
        x = x.double()
        z = x[..., :rot].unflatten(-1, (rot // 2, 2) if s["interleaved"] else (2, rot // 2))
        z = z if s["interleaved"] else z.transpose(-1, -2)
        turns = torch.polar(torch.full_like(s["inv"], s["multiplier"]).expand(len(where), -1), where[:, None] * s["inv"])
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turns[:, None])
        return torch.cat([(z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., rot:]], -1)

    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)

    def rounded(x):  # the value that the row's codes and scales stand for
        b = x.float().double().unflatten(-1, (-1, 16))
        scale = (b.abs().amax(-1).float() / 6).clamp(max=448).to(E4M3).double()[..., None]
        q = torch.where(scale > 0, b / scale.clamp(min=1e-300), 0.0)
        away = (q.abs()[..., None] - grid).abs()
        # the nearest of the grid, of two at the same distance the one with the even code
        away = away - 1e-12 * (1 - torch.arange(8, device=DEV) % 2)
        return (grid[away.argmin(-1)] * torch.sign(q) * scale).flatten(-2)

    pools = {}
    for x in ("k", "v"):
        every = torch.arange(s["batch"]["pages"], device=DEV)
        pools[x] = torch.stack([_decoded(s, x, every, h).view(len(every), page, -1) for h in range(s["kv_heads"])], 1)
    qs = []
    for r, (n, kv) in enumerate(zip(news, kvs)):
        slot = torch.arange(kv - n, kv)
        where = slot.double().to(DEV) if s["positions"] is None else s["positions"][at: at + n].double()
        qs.append(turn(s["q"][at: at + n], where))
        ids, row = table[r, slot // page].to(DEV), (slot % page).to(DEV)
        pools["k"][ids, :, row] = rounded(turn(s["new_k"][at: at + n], where))
        pools["v"][ids, :, row] = rounded(s["new_v"][at: at + n])
        at += n
    return dict(q=torch.cat(qs), **pools)


def _drafts_exact(s, news):
    """Request by request, draft by draft."""
    accepted, out, at, drawn = [], [], 0, 0
    for r, n in enumerate(news):
        rows = s["target"][at: at + n].double()
        if s["given"] == "logits":
            if s["temperature"][r] == 0:
                best = torch.nonzero(rows == rows.max(1, keepdim=True).values)
                p = torch.zeros_like(rows)
                for i in range(n):
                    p[i, best[best[:, 0] == i][0, 1]] = 1.0
            else:
                p = torch.softmax(rows * (1.0 / s["temperature"][r].double()), 1)
        else:
            p = rows
        ids, count = s["ids"][at + 1: at + n].tolist(), 0
        q = None
        while count < n - 1:
            q = s["draft"][drawn + count].double() if s["draft"] is not None else \
                torch.nn.functional.one_hot(torch.tensor(ids[count], device=DEV), s["vocab"]).double()
            if float(s["u_accept"][at + count]) * float(q[ids[count]]) >= float(p[count, ids[count]]):
                break
            count += 1
        w = p[count]
        if count < n - 1:
            less = torch.relu(w - q) if s["draft"] is not None else w * (1 - q)
            w = less if float(less.sum()) > 0 else w
        c = torch.cumsum(w, 0)
        nxt = torch.nonzero(c > float(s["u_next"][r]) * c[-1])
        nxt = int(nxt[0]) if len(nxt) else int(torch.nonzero(w > 0)[-1])
        accepted.append(count)
        out += ids[:count] + [nxt] + [-1] * (n - 1 - count)
        at, drawn = at + n, drawn + n - 1
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(accepted=whole(accepted), out=whole(out))
