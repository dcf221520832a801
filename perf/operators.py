"""Cases of the operators around the MLP block of a speculative-verify layer, with their plain forms.

* norm: residual addition + RMSNorm, with an E4M3 output (codes, one scale per token) and / or a bf16 one
* rope: rotary positions of q and k, and the append of k and v to a paged cache (bf16, or E4M3 with scales)
* attn: attention of each request's new tokens over its paged cache, with an optional sliding window and first
  tokens that stay visible

A batch is `requests` requests; request r brings n_r new tokens (`mix`: all `new`, or spread) and has kv_r tokens in
the cache when these are in it.  Both follow from the case alone, so that work() counts exactly what is read.
"""

import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of one request entering a layer: latency
        dict(name="norm_one", op="norm", rows=1, hidden=2048, residual=True, codes=True, plain=False),
        # the verify pass of 16 requests x (1 + 12 drafts) in front of the MLP block
        dict(name="norm_verify", op="norm", rows=208, hidden=4096, residual=True, codes=True, plain=False),
        # a prompt's tokens, the bf16 output for the projections beside the 8-bit one
        dict(name="norm_prompt", op="norm", rows=8191, hidden=4096, residual=True, codes=True, plain=True),
        # one request decoding, bf16 cache: latency
        dict(name="rope_one", op="rope", requests=1, new=1, kv=333, mix="even", heads=16, kv_heads=4, dim=128, rot=128,
             page=16, e4m3=False, interleaved=False, scaling="none", offset=0),
        # the verify pass into an E4M3 cache, positions scaled for a longer context
        dict(name="rope_verify_e4m3", op="rope", requests=16, new=13, kv=2000, mix="even", heads=32, kv_heads=8,
             dim=128, rot=128, page=64, e4m3=True, interleaved=False, scaling="yarn", offset=0),
        # prompts of uneven lengths, half of each head rotated, interleaved pairs, positions far from zero
        dict(name="rope_prompt", op="rope", requests=4, new=2048, kv=2500, mix="ragged", heads=32, kv_heads=8, dim=128,
             rot=64, page=64, e4m3=False, interleaved=True, scaling="linear", offset=1000003),
        # the smallest call: one short request, one token
        dict(name="attn_one", op="attn", requests=1, new=1, kv=257, mix="even", heads=16, kv_heads=4, dim=128, page=16,
             e4m3=False, window=0, sinks=0),
        # the verify pass: 16 requests x 13 rows over uneven contexts
        dict(name="attn_verify", op="attn", requests=16, new=13, kv=4096, mix="contexts", heads=32, kv_heads=8,
             dim=128, page=64, e4m3=False, window=0, sinks=0),
        # a large verify batch over an E4M3 cache
        dict(name="attn_verify_e4m3", op="attn", requests=64, new=13, kv=8192, mix="contexts", heads=32, kv_heads=8,
             dim=128, page=64, e4m3=True, window=0, sinks=0),
        # long contexts, one token each: the cache is all there is to read
        dict(name="attn_long", op="attn", requests=4, new=1, kv=131072, mix="contexts", heads=32, kv_heads=8, dim=128,
             page=64, e4m3=False, window=0, sinks=0),
        # chunks of two prompts after earlier chunks: matrix-core work
        dict(name="attn_chunk", op="attn", requests=2, new=2048, kv=10007, mix="ragged", heads=32, kv_heads=8, dim=128,
             page=64, e4m3=False, window=0, sinks=0),
        # a sliding-window layer with four first tokens kept, small heads
        dict(name="attn_window", op="attn", requests=32, new=13, kv=16384, mix="contexts", heads=16, kv_heads=4, dim=64,
             page=32, e4m3=False, window=1024, sinks=4),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    if op == "norm":
        hidden = 8 * _spread(rng, 16, 2048)
        rows = min(_spread(rng, 1, 8192), max(1, (1 << 25) // hidden))
        codes = rng.random() < 0.75
        return dict(op="norm", rows=rows, hidden=hidden, residual=rng.random() < 0.75, codes=codes,
                    plain=not codes or rng.random() < 0.3)
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8])
    page, e4m3 = rng.choice([16, 32, 64, 128]), rng.random() < 0.5
    requests, mix = _spread(rng, 1, 64), rng.choice(["even", "contexts", "ragged"])
    new = rng.choice([1, _spread(rng, 2, 16), _spread(rng, 16, 2048)])
    if op == "rope":
        new = min(new, max(1, (1 << 25) // (requests * (heads + 2 * kv_heads) * dim)))
        kv = new + min(_spread(rng, 1, 4096), max(1, (1 << 25) // (requests * kv_heads * dim)))
        return dict(op="rope", requests=requests, new=new, kv=kv, mix=mix, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), page=page, e4m3=e4m3, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), offset=rng.choice([0, 0, 70001, 1000003]))
    # no more cache, scores or products than the listed cases have
    new = min(new, max(1, (1 << 24) // (requests * heads)))
    most = min((1 << 29) // (requests * kv_heads * dim), (1 << 30) // (requests * heads * new),
               (1 << 37) // (requests * heads * new * dim))
    kv = new + min(_spread(rng, 1, 131072), max(1, most - new))
    window = rng.choice([0, 0, _spread(rng, 16, 4096)])
    return dict(op="attn", requests=requests, new=new, kv=kv, mix=mix, heads=heads, kv_heads=kv_heads, dim=dim,
                page=page, e4m3=e4m3, window=window, sinks=rng.choice([0, 1, 4, 17]) if window else 0)


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each request."""
    n, kv, requests, mix = case["new"], case["kv"], case["requests"], case["mix"]
    news = [n if mix != "ragged" or r == 0 else max(1, n - (r * n * 29 // 64) % n) for r in range(requests)]
    kvs = [kv if mix == "even" or r == 0 else max(news[r], kv - (r * kv * 37 // 100) % (kv // 2 + 1))
           for r in range(requests)]
    return news, kvs


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
    return inv * keep + inv / factor * (1 - keep), 0.1 * math.log(factor) + 1


def _quantized(x):
    """E4M3 codes and scales (amax / 448) over the last axis."""
    scale = x.abs().amax(-1) / 448.0
    q = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return q.clamp(-448, 448).to(E4M3), scale


def _filled(shape, e4m3, gen):
    """A cache's pool [pages, kv_heads, page, dim] with what earlier steps left in it, and its scales."""
    x = torch.randn(shape, device=DEV, generator=gen, dtype=torch.float32 if e4m3 else torch.bfloat16)
    return _quantized(x) if e4m3 else (x, None)


def _batch(case, gen):
    news, kvs = _lengths(case)
    page, requests = case["page"], case["requests"]
    most = max(-(-kv // page) for kv in kvs)
    pages = requests * most
    start = [0]
    for n in news:
        start.append(start[-1] + n)
    table = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32).reshape(requests, most)
    return dict(start=torch.tensor(start, dtype=torch.int32, device=DEV),
                kv=torch.tensor(kvs, dtype=torch.int32, device=DEV), table=table, max_new=max(news), max_kv=max(kvs),
                tokens=start[-1], pages=pages)


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, device=DEV, generator=gen).to(torch.bfloat16)  # noqa: E731
    s = dict(case)
    if case["op"] == "norm":
        rows, hidden = case["rows"], case["hidden"]
        x = torch.randn((rows, hidden), device=DEV, generator=gen)
        x[:, torch.randperm(hidden, device=DEV, generator=gen)[: max(1, hidden // 100)]] *= 20  # outlier channels
        s["x"] = x.to(torch.bfloat16)
        s["res"] = randn(rows, hidden) * 3 if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(hidden, device=DEV, generator=gen)).to(torch.bfloat16)
        return s
    b = s["batch"] = _batch(case, gen)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    pool = (b["pages"], kv_heads, case["page"], dim)
    s["k"], s["ks"] = _filled(pool, case["e4m3"], gen)
    s["v"], s["vs"] = _filled(pool, case["e4m3"], gen)
    if case["op"] == "rope":
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
        s["own_cache"] = ocq.PagedKVCache(s["k"], s["v"], s["ks"], s["vs"])
        s["own_batch"] = ocq.TokenBatch(b["start"], b["kv"], b["table"], b["max_new"], b["max_kv"])
        if case["op"] == "rope":
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


def _norm_plain(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    out = {}
    if s["res"] is not None:
        out["residual"] = h.to(torch.bfloat16)
    if s["plain"]:
        out["y"] = y.to(torch.bfloat16)
    if s["codes"]:
        out["codes"], out["scales"] = _quantized(y)
    return out


def _rotated(x, cos, sin, s):
    rot = s["rot"]
    y = x.float()
    if s["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _rope_plain(s):
    r, _ = _request_of(s)
    place = _positions(s)
    angle = (place if s["positions"] is None else s["positions"]).double()[:, None] * s["inv"]
    cos, sin = ((f(angle) * s["multiplier"]).float()[:, None] for f in (torch.cos, torch.sin))
    q = _rotated(s["q"], cos, sin, s).to(torch.bfloat16)
    k, v = _rotated(s["new_k"], cos, sin, s), s["new_v"].float()
    page, row = s["batch"]["table"][r, place // s["page"]].long(), place % s["page"]
    if s["e4m3"]:
        (k, ks), (v, vs) = _quantized(k), _quantized(v)
        s["k"].view(torch.uint8)[page, :, row] = k.view(torch.uint8)
        s["v"].view(torch.uint8)[page, :, row] = v.view(torch.uint8)
        s["ks"][page, :, row], s["vs"][page, :, row] = ks, vs
    else:
        s["k"][page, :, row], s["v"][page, :, row] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return dict(q=q, **_cache_of(s))


def _cache_of(s):
    return {n: s[n] for n in ("k", "v", "ks", "vs") if s[n] is not None}


def _gathered(pool, scales, table):
    """[requests, kv_heads, tokens, dim] in 32 bits out of the pages."""
    x = (pool.view(torch.uint8)[table].view(E4M3) if scales is not None else pool[table]).float()
    if scales is not None:
        x = x * scales[table][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _attn_plain(s):
    b, heads, kv_heads, dim = s["batch"], s["heads"], s["kv_heads"], s["dim"]
    group, requests, n = heads // kv_heads, s["requests"], b["max_new"]
    k, v = (_gathered(s[x], s[x + "s"], b["table"].long()) for x in ("k", "v"))
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


def _run_own(s):
    from quantized_memory_bound_amd import ocq
    if s["op"] == "norm":
        residual, y, codes, scales = ocq.add_rmsnorm(s["x"], s["w"], eps=1e-6, residual=s["res"], want_y=s["plain"],
                                                     want_codes=s["codes"])
        out = dict(residual=residual, y=y, codes=codes, scales=scales)
        return {k: v for k, v in out.items() if v is not None}
    if s["op"] == "rope":
        q = ocq.rope_append(s["q"], s["new_k"], s["new_v"], s["own_rope"], s["own_cache"], s["own_batch"],
                            positions=s["positions"])
        return dict(q=q, **_cache_of(s))
    out, lse = ocq.paged_attention(s["q"], s["own_cache"], s["own_batch"], window=s["window"], sinks=s["sinks"],
                                   want_lse=True)
    return dict(out=out, lse=lse)


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm_plain, "rope": _rope_plain, "attn": _attn_plain}[s["op"]](s)


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["hidden"]
        out = n * (2 * case["residual"] + 2 * case["plain"] + case["codes"]) + 4 * case["rows"] * case["codes"]
        return dict(bytes=n * (2 + 2 * case["residual"]) + 2 * case["hidden"] + out, flops=8 * n)
    news, kvs = _lengths(case)
    heads, kv_heads, dim, tokens = case["heads"], case["kv_heads"], case["dim"], sum(news)
    row = kv_heads * (dim + 4 if case["e4m3"] else 2 * dim)  # cached bytes of one token's k (or v)
    if case["op"] == "rope":
        return dict(bytes=tokens * (2 * (heads + 2 * kv_heads) * dim + 2 * heads * dim + 2 * row),
                    flops=3 * tokens * (heads + kv_heads) * case["rot"])
    window, sinks, read, pairs = case["window"], case["sinks"], 0, 0
    for n, kv in zip(news, kvs):
        first = kv - n                                            # place of the first new token
        low = max(0, first - window + 1) if window else 0
        read += kv - low + min(sinks if window else 0, low)       # tokens that some row sees
        if window:
            pairs += sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(first, kv))
        else:
            pairs += n * first + n * (n + 1) // 2
    return dict(bytes=2 * row * read + tokens * heads * (4 * dim + 4) + 4 * (read // case["page"]),
                flops=4 * dim * heads * pairs)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0)
        y = s["w"].double() * h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + 1e-6)
        scale = y.abs().max(1).values / 448
        out = dict(residual=h if case["residual"] else None, y=y if case["plain"] else None)
        if case["codes"]:  # the quotient that a code rounds
            out |= dict(codes=y / scale.clamp(min=1e-300)[:, None], scales=scale)
        return out
    news, kvs = _lengths(case)
    table, page = s["batch"]["table"].long().cpu(), case["page"]
    if case["op"] == "rope":
        return _rope_exact(s, news, kvs, table, page)
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
            k, v = ((s[x].view(torch.uint8)[ids, h].view(E4M3).double() * s[x + "s"][ids, h].double()[..., None]
                     if case["e4m3"] else s[x][ids, h].double()).reshape(-1, case["dim"])[:kv] for x in ("k", "v"))
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


def _rope_exact(s, news, kvs, table, page):
    rot, at = s["rot"], 0

    def turn(x, where):  # pairs as complex numbers, turned by e^(i angle)
        x = x.double()
        z = x[..., :rot].unflatten(-1, (rot // 2, 2) if s["interleaved"] else (2, rot // 2))
        z = z if s["interleaved"] else z.transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.full_like(s["inv"], s["multiplier"]).expand(len(where), -1),
                                                                where[:, None] * s["inv"])[:, None]
        z = torch.view_as_real(z)
        return torch.cat([(z if s["interleaved"] else z.transpose(-1, -2)).flatten(-2), x[..., rot:]], -1)

    cache = {x: s[x].double() for x in ("k", "v", "ks", "vs") if s[x] is not None}
    qs = []
    for r, (n, kv) in enumerate(zip(news, kvs)):
        slot = torch.arange(kv - n, kv)
        where = slot.double().to(DEV) if s["positions"] is None else s["positions"][at: at + n].double()
        qs.append(turn(s["q"][at: at + n], where))
        ids, row = table[r, slot // page].to(DEV), (slot % page).to(DEV)
        for x, y in (("k", turn(s["new_k"][at: at + n], where)), ("v", s["new_v"][at: at + n].double())):
            if s["e4m3"]:
                scale = y.abs().max(-1).values / 448
                cache[x + "s"][ids, :, row] = scale
                y = y / scale.clamp(min=1e-300)[..., None]  # the quotient that a code rounds
            cache[x][ids, :, row] = y
        at += n
    return dict(q=torch.cat(qs), **cache)
