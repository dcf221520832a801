"""One layer of a speculative-verify step: attention over a paged cache and the quantized MLP block.

    python -m quantized_memory_bound_amd.verify_layer [--requests 16 --drafts 12 --context 4000 --e4m3 | --nvfp4] [--loop]

The verify pass checks 1 + drafts tokens of every request at once ("Generate more tokens per target pass: speculative
decoding" in the post).  A layer is

    x, h = norm(x + attention output of the layer before ...)         ocq.add_rmsnorm
    q, k, v = h Wqkv                                                  a library product (bf16)
    q, cache <- rotary positions, append                              ocq.rope_append
    o = attention of the new tokens over the cache                    ocq.paged_attention
    x, h = norm(x + o Wo)                                             ocq.add_rmsnorm
    m = MLP block(h), added to x by the next layer's norm             ocq.mlp_forward

Rejected drafts cost nothing: the next step's kv_lens count only what was accepted, and its tokens overwrite the rest.

VerifyLoop closes the step on the GPU: which drafts the target accepts and the token after them (ocq.verify_drafts), and
the next step's offsets, lengths and pages (ocq.step_tables), without a word to the host (--loop times it).
"""

import argparse
import time

import numpy as np

from . import ocq


class VerifyLayer:
    """Weights, cache and workspace of one layer, for repeated steps.

    w_qkv: bf16 [hidden, (heads + 2 kv_heads) * head_dim], w_o: bf16 [heads * head_dim, hidden], norm_in, norm_mlp:
    bf16 [hidden] (CUDA); mlp: an ocq.QuantizedMLP; cache: an ocq.PagedKVCache; rope: an ocq.Rope.
    """

    def __init__(self, heads, w_qkv, w_o, norm_in, norm_mlp, mlp, cache, rope, eps=1e-6, window=0, sinks=0):
        self.heads, self.cache, self.rope, self.mlp = heads, cache, rope, mlp
        self.w_qkv, self.w_o, self.norm_in, self.norm_mlp = w_qkv, w_o, norm_in, norm_mlp
        self.eps, self.window, self.sinks = eps, window, sinks

    def __call__(self, x, pending, batch):
        """x: bf16 [tokens, hidden], the residual stream; pending: what the layer before left to add to it (None in
        the first layer).  Returns (x, pending) for the next layer."""
        c = self.cache
        new_x, h, _, _ = ocq.add_rmsnorm(x, self.norm_in, self.eps, residual=pending, want_y=True, want_codes=False)
        x = x if pending is None else new_x
        qkv = (h @ self.w_qkv).view(x.shape[0], self.heads + 2 * c.kv_heads, c.head_dim)
        q, k, v = qkv.split([self.heads, c.kv_heads, c.kv_heads], 1)
        q = ocq.rope_append(q, k, v, self.rope, c, batch)
        o, _ = ocq.paged_attention(q, c, batch, window=self.window, sinks=self.sinks)
        x, h, _, _ = ocq.add_rmsnorm(x, self.norm_mlp, self.eps, residual=o.flatten(1) @ self.w_o, want_y=True,
                                     want_codes=False)
        return x, self.mlp(h)


class VerifyLoop:
    """Speculative decoding of a batch over one layer: embed, layer, head, and everything between two steps on the GPU.

    layer: a VerifyLayer; embed: bf16 [vocab, hidden]; head: bf16 [hidden, vocab]; tables: ocq.PageTables of empty
    requests over the layer's cache; drafts: drafted tokens a request and step; max_kv: a host bound of any request's
    tokens in the cache.  The draft model is the embedding and the head without the layer: each draft is drawn from
    softmax(embed[token before] head / temperature), or is its largest logit where temperature, a number, is 0.

    missing: int64 [1], the pages that steps lacked, summed over them (tokens without a page are lost to the steps that
    follow; the host looks at it when it likes).
    """

    def __init__(self, layer, embed, head, tables, drafts, max_kv, temperature=1.0, seed=0):
        import torch
        self.layer, self.embed, self.head, self.tables = layer, embed, head, tables
        self.drafts, self.max_kv, self.temperature = drafts, max_kv, float(temperature)
        if not 0 <= self.temperature < float("inf"):
            raise ocq.OcqError(ocq.ERR_INVALID_ARG, "temperature must be finite and not negative, got %g" % self.temperature)
        dev, requests = tables.device, tables.requests
        self.gen = torch.Generator(dev).manual_seed(seed)
        self.batch = ocq.TokenBatch(tables.q_start, tables.kv_lens, tables.page_table, 1 + drafts, max_kv,
                                    tokens=requests * (1 + drafts))
        self.news = torch.full((requests,), 1 + drafts, dtype=torch.int32, device=dev)
        self.first = torch.arange(requests, device=dev) * (1 + drafts)
        self.accepted = None          # all of the prompt's tokens stay
        self.last = None
        self.missing = torch.zeros(1, dtype=torch.int64, device=dev)

    def prefill(self, prompts, chunk=512):
        """prompts: int [requests, length]; all but their last tokens go into the cache, behind what steps before have
        left there (the token that such a step ended with, `last`, is not in it yet).  Raises where the cache has not
        enough pages for them (this waits for the GPU; it then holds a part of the prompts)."""
        import torch
        requests, length = prompts.shape
        lacking = torch.zeros_like(self.missing)
        for at in range(0, length - 1, chunk):
            ids = prompts[:, at: min(at + chunk, length - 1)]
            n = ids.shape[1]
            lacking += ocq.step_tables(self.tables, torch.full_like(self.news, n), requests * n, accepted=self.accepted)[3]
            self.accepted = None
            batch = ocq.TokenBatch(self.tables.q_start, self.tables.kv_lens, self.tables.page_table, n, at + n)
            self.layer(self.embed[ids.flatten()], None, batch)
        if int(lacking):
            raise ocq.OcqError(ocq.ERR_BUFFER_TOO_SMALL, "prompts of %d tokens: the cache has too few pages for them, or "
                               "max_pages is too small" % length)
        self.last = prompts[:, -1].to(torch.int32)

    def step(self):
        """One verify step: (accepted int32 [requests], out int32 [requests, 1 + drafts], each request's accepted
        drafts, the next token and -1).  A request whose next token was -1 (its logits are not numbers) has ended: it
        takes part with token 0, of which nothing stays in the cache, and its row is -1, until the next prefill."""
        import torch
        requests, vocab = self.tables.requests, self.head.shape[1]

        def rand(*shape):
            return torch.rand(shape, device=self.last.device, generator=self.gen)
        ended = self.last < 0
        ids, probs = [self.last.clamp(min=0)], []
        for _ in range(self.drafts):
            logits = (self.embed[ids[-1]] @ self.head).float()
            if self.temperature == 0:             # not drawn: no probabilities to compare with
                ids.append(logits.argmax(-1).to(torch.int32))
                continue
            probs.append(torch.softmax(logits / self.temperature, -1))
            ids.append((probs[-1] / -torch.log(rand(requests, vocab).clamp(min=1e-30))).argmax(-1).to(torch.int32))
        ids = torch.stack(ids, 1).flatten()
        self.missing += ocq.step_tables(self.tables, self.news, len(ids), accepted=self.accepted)[3]
        x, pending = self.layer(self.embed[ids], None, self.batch)
        accepted, out = ocq.verify_drafts((x + pending) @ self.head, ids, self.batch, rand(len(ids)), rand(requests),
                                          draft_probs=torch.stack(probs, 1).flatten(0, 1) if probs else None,
                                          temperature=self.temperature)
        out.view(requests, -1).masked_fill_(ended[:, None], -1)
        accepted.masked_fill_(ended, 0)
        self.last = out[self.first + accepted]
        self.accepted = accepted - ended.to(torch.int32)     # -1: not even the first token stays
        return accepted, out.view(requests, -1)


def random_layer(hidden, inter, heads, kv_heads, head_dim, pages, page_size, e4m3=False, seed=0, device="cuda",
                 prec_mode=ocq.PREC_FP8, nvfp4=False, **kw):
    """A layer of random weights over an empty cache."""
    import torch
    gen = torch.Generator(device).manual_seed(seed)

    def rand(*shape, std):
        return (torch.randn(shape, device=device, generator=gen) * std).to(torch.bfloat16)
    rng = np.random.default_rng(seed)
    w = [rng.standard_normal(s, dtype=np.float32) * np.float32(0.02)
         for s in ((inter, hidden), (inter, hidden), (hidden, inter))]
    cache = ocq.PagedKVCache.allocate(pages, page_size, kv_heads, head_dim, e4m3, device, nvfp4)
    return VerifyLayer(heads, rand(hidden, (heads + 2 * kv_heads) * head_dim, std=hidden ** -0.5),
                       rand(heads * head_dim, hidden, std=0.02), 1 + rand(hidden, std=0.1), 1 + rand(hidden, std=0.1),
                       ocq.QuantizedMLP(*w, prec_mode, device), cache, ocq.Rope.make(head_dim, device=device), **kw)


def batch_of(news, kv_lens, page_table, device="cuda"):
    """The TokenBatch of host lists: new tokens and cached tokens of each request, and its pages."""
    import torch
    start = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32).to(device)
    return ocq.TokenBatch(start, torch.tensor(kv_lens, dtype=torch.int32).to(device), page_table, max(1, max(news)),
                          max(kv_lens))


def main():
    import torch
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--drafts", type=int, default=12)
    ap.add_argument("--context", type=int, default=4000)
    ap.add_argument("--e4m3", action="store_true", help="E4M3 cache")
    ap.add_argument("--nvfp4", action="store_true", help="NVFP4 cache")
    ap.add_argument("--loop", action="store_true", help="whole steps: drafts, tables, layer, head, verification")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    hidden, inter, heads, kv_heads, dim, page = 2048, 6144, 16, 4, 128, 64
    n = 1 + a.drafts
    per = -(-(a.context + n * (a.steps + 2)) // page)
    layer = random_layer(hidden, inter, heads, kv_heads, dim, a.requests * per, page, a.e4m3, nvfp4=a.nvfp4)
    cached = "E4M3" if a.e4m3 else "NVFP4" if a.nvfp4 else "bf16"
    if a.loop:
        return time_loop(layer, a, a.requests * per, page, cached)
    table = torch.randperm(a.requests * per).to(torch.int32).view(a.requests, per).cuda()
    gen = torch.Generator("cuda").manual_seed(1)

    def rows(count):
        return torch.randn((count, hidden), device="cuda", generator=gen).to(torch.bfloat16)
    chunk, done = 512, 0
    while done < a.context:                                     # the prompts, in chunks
        c = min(chunk, a.context - done)
        done += c
        layer(rows(a.requests * c), None, batch_of([c] * a.requests, [done] * a.requests, table))
    x, rng, lens = rows(a.requests * n), np.random.default_rng(0), [a.context] * a.requests
    spent = 0.0
    for step in range(a.steps + 2):
        batch = batch_of([n] * a.requests, [l + n for l in lens], table)
        torch.cuda.synchronize()
        t = time.perf_counter()
        out, pending = layer(x, None, batch)
        torch.cuda.synchronize()
        spent += time.perf_counter() - t if step >= 2 else 0.0
        assert torch.isfinite(out.float()).all() and torch.isfinite(pending.float()).all()
        lens = [l + 1 + int(rng.integers(0, a.drafts + 1)) for l in lens]     # accepted tokens stay, the rest goes
    print("verify layer: %d requests x %d tokens, contexts of %d to %d tokens (%s cache): %.1f us a step" %
          (a.requests, n, min(lens), max(lens), cached, spent / a.steps * 1e6))


def time_loop(layer, a, pages, page, cached, vocab=32768):
    import torch
    gen = torch.Generator("cuda").manual_seed(2)

    def rand(*shape, std):
        return (torch.randn(shape, device="cuda", generator=gen) * std).to(torch.bfloat16)
    hidden = layer.w_qkv.shape[0]
    tables = ocq.PageTables.allocate(a.requests, pages // a.requests, pages, page)
    loop = VerifyLoop(layer, rand(vocab, hidden, std=1.0), rand(hidden, vocab, std=2.0 * hidden ** -0.5), tables, a.drafts,
                      pages // a.requests * page)
    loop.prefill(torch.randint(0, vocab, (a.requests, a.context + 1), device="cuda", generator=gen))
    kept, t = 0, 0.0
    for step in range(a.steps + 2):
        if step == 2:
            torch.cuda.synchronize()
            t, kept = time.perf_counter(), 0
        accepted, _ = loop.step()
        kept = kept + accepted.sum() + a.requests
    torch.cuda.synchronize()
    spent = time.perf_counter() - t
    assert int(loop.missing) == 0
    print("verify loop: %d requests x %d tokens, contexts of %d to %d tokens (%s cache), vocabulary %d: %.1f us a step, "
          "%.2f tokens a request and step" % (a.requests, 1 + a.drafts, int(tables.kv_lens.min()), int(tables.kv_lens.max()),
                                              cached, vocab, spent / a.steps * 1e6, int(kept) / a.steps / a.requests))


if __name__ == "__main__":
    main()
