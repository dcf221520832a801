"""One layer of a speculative-verify step: attention over a paged cache and the quantized MLP block.

    python -m quantized_memory_bound_amd.verify_layer [--requests 16 --drafts 12 --context 4000 --e4m3]

The verify pass checks 1 + drafts tokens of every request at once ("Generate more tokens per target pass: speculative
decoding" in the post).  A layer is

    x, h = norm(x + attention output of the layer before ...)         ocq.add_rmsnorm
    q, k, v = h Wqkv                                                  a library product (bf16)
    q, cache <- rotary positions, append                              ocq.rope_append
    o = attention of the new tokens over the cache                    ocq.paged_attention
    x, h = norm(x + o Wo)                                             ocq.add_rmsnorm
    m = MLP block(h), added to x by the next layer's norm             ocq.mlp_forward

Rejected drafts cost nothing: the next step's kv_lens count only what was accepted, and its tokens overwrite the rest.
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


def random_layer(hidden, inter, heads, kv_heads, head_dim, pages, page_size, e4m3=False, seed=0, device="cuda",
                 prec_mode=ocq.PREC_FP8, **kw):
    """A layer of random weights over an empty cache."""
    import torch
    gen = torch.Generator(device).manual_seed(seed)

    def rand(*shape, std):
        return (torch.randn(shape, device=device, generator=gen) * std).to(torch.bfloat16)
    rng = np.random.default_rng(seed)
    w = [rng.standard_normal(s, dtype=np.float32) * np.float32(0.02)
         for s in ((inter, hidden), (inter, hidden), (hidden, inter))]
    cache = ocq.PagedKVCache.allocate(pages, page_size, kv_heads, head_dim, e4m3, device)
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
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    hidden, inter, heads, kv_heads, dim, page = 2048, 6144, 16, 4, 128, 64
    n = 1 + a.drafts
    per = -(-(a.context + n * (a.steps + 2)) // page)
    layer = random_layer(hidden, inter, heads, kv_heads, dim, a.requests * per, page, a.e4m3)
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
          (a.requests, n, min(lens), max(lens), "E4M3" if a.e4m3 else "bf16", spent / a.steps * 1e6))


if __name__ == "__main__":
    main()
