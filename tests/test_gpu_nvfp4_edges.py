"""Attention over NVFP4 caches at its ends: rows of q next to zero, scales and units that meet them, contexts longer than the
caller's bound.  References and tolerances are those of test_gpu_nvfp4_cache.py."""

import math

import pytest
import torch

from quantized_memory_bound_amd import ocq
from test_gpu_layer import _bf, _gen, make_batch
from test_gpu_nvfp4_cache import attention_ref, check_attention, make_cache, rows_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 13, 40, 300])
@pytest.mark.parametrize("size,unit,scale", [
    (2.0 ** -80, 2.0 ** -64, None),       # scale x unit x max |q| below 2^-140: every score is 0 in 32 bits
    (2.0 ** -133, 1.0, None),             # bf16's smallest numbers
    (1.0, 2.0 ** -64, 2.0 ** -90), (2.0 ** -100, 1.0, 2.0 ** -60),
    (2.0 ** 100, 2.0 ** -64, 2.0 ** -80),  # scale x unit alone is below 2^-126, the scores are not small
    (2.0 ** -133, 2.0 ** 64, 2.0 ** 65),   # scale x unit alone is past 2^128
    (0.0, 2.0 ** 64, 2.0 ** 80)])
def test_attention_rows_next_to_zero(dim, n, size, unit, scale):
    """Causal and window edges, where masked scores are -inf; 300 rows of four heads are widened first."""
    g = _gen(dim + n)
    news, kvs = [n, 1], [n + 310, 777]
    batch, pages = make_batch(news, kvs, 16, g)
    cache = make_cache(pages, 1, 16, dim, g, units=(unit, 1.0))
    q = (torch.randint(-3, 4, (sum(news), 4, dim), device=DEV, generator=g).double() * size).to(torch.bfloat16)
    q[0, 0] = 0
    check_attention(q, cache, batch, news, kvs, scale=scale)
    check_attention(q, cache, batch, news, kvs, scale=scale, window=100, sinks=3)


def limited_ref(q, cache, batch, news, kvs, window, sinks, limit):
    """Tokens at the places that kv_lens give them, over the keys below limit alone."""
    out, lse, mag, at = [], [], [], 0
    group = q.shape[1] // cache.kv_heads
    for r, (n, kv) in enumerate(zip(news, kvs)):
        qq = q[at: at + n].double().transpose(0, 1).contiguous()
        at += n
        j = torch.arange(min(kv, limit), device=DEV)
        p = torch.arange(kv - n, kv, device=DEV)
        seen = j[None] <= p[:, None]
        if window:
            seen = seen & ((j[None] > p[:, None] - window) | (j[None] < sinks))
        k, v = (rows_of(cache, w, batch.page_table[r], j).repeat_interleave(group, 1).permute(1, 0, 2).contiguous()
                for w in ("k", "v"))
        s = torch.matmul(qq, k.transpose(1, 2).contiguous()) * q.shape[2] ** -0.5
        s = s.masked_fill(~seen[None], -math.inf)
        some = seen.any(-1)
        w = torch.where(some[None, :, None], torch.softmax(s, -1), torch.zeros_like(s))
        out.append(torch.matmul(w, v).transpose(0, 1))
        lse.append(torch.logsumexp(s, -1).transpose(0, 1))
        both = [torch.matmul(x, v.abs()) for x in (w, seen[None].expand(len(w), -1, -1).double())]
        mag.append(torch.stack(both).transpose(1, 2))
    return torch.cat(out), torch.cat(lse), torch.cat(mag, 1)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (333, 0), (100, 130)])
@pytest.mark.parametrize("limit", [1, 500, 1024, 1999])
def test_attention_contexts_longer_than_max_kv(dim, page, window, sinks, limit):
    """Calls whose pages are widened first, with a max_kv that some contexts are past: every token keeps its place, tokens
    whose place is below max_kv are as ever, the others see the keys below it."""
    g = _gen(dim + limit)
    news, kvs = [700, 5, 300], [1500, 2100, 300]
    batch, pages = make_batch(news, kvs, page, g)
    cache = make_cache(pages, 2, page, dim, g, "tokens", (0.25, 2.0 ** 5))
    short = ocq.TokenBatch(batch.q_start, batch.kv_lens, batch.page_table, 700, limit)
    q = _bf((sum(news), 8, dim), g)
    out, lse = ocq.paged_attention(q, cache, short, window=window, sinks=sinks, want_lse=True)
    ref, rl, mag = limited_ref(q, cache, batch, news, kvs, window, sinks, limit)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and not out[empty].float().any()
    d = (lse.double() - rl)[~empty].abs()
    assert not d.numel() or d.max() <= 2.0 ** -18 + rl[~empty].abs().max() * 2.0 ** -18
    tol = ref.abs() * 2.0 ** -8 + mag[0] * (2.0 ** -11 + 2.0 ** -14) + mag[1] * 2.0 ** -32 + 1e-30
    assert ((out.double() - ref).abs() <= tol).all()
    # the definition itself, where max_kv cuts nothing off
    full, _, m = attention_ref(q, cache, batch, news, kvs, dim ** -0.5, window, sinks)
    places = torch.cat([torch.arange(kv - n, kv, device=DEV) for n, kv in zip(news, kvs)])
    ok = places < limit
    assert ((out.double() - full).abs() <= full.abs() * 2.0 ** -8 + m[0] * (2.0 ** -11 + 2.0 ** -14) + m[1] * 2.0 ** -32 +
            1e-30)[ok].all()
