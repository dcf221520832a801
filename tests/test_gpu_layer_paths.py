"""Paths of the operators around the block that only some sizes take, and what has to agree to the bit: one append of
many tokens with many of one, and the layer's MLP half with the block.  Tolerances as in test_gpu_layer.py."""

import numpy as np
import pytest
import torch

from oracle import mlp as O
from parity import check_y
from quantized_memory_bound_amd import ocq
from quantized_memory_bound_amd.verify_layer import batch_of, random_layer
from test_gpu_layer import (DEV, _bf, _check_bf16, _check_codes, _gen, _norm_ref, check_attention, make_batch,
                            make_cache)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norm of inputs far larger than the caches

@pytest.mark.parametrize("rows,hidden", [(32771, 512), (8195, 2048), (4097, 4096), (2049, 8192), (1025, 16384),
                                         (514, 32768), (257, 65536)])
def test_norm_of_more_than_2_24_values(rows, hidden):
    g = _gen(rows)
    x, res, w = _bf((rows, hidden), g, 2.0), _bf((rows, hidden), g), _bf((hidden,), g)
    r, y, c, s = ocq.add_rmsnorm(x, w, 1e-5, residual=res, want_y=True)
    h, ref = _norm_ref(x, w, 1e-5, res)
    size = x.double().abs() + res.double().abs()
    _check_bf16(r, h, "residual", extra=size * 2.0 ** -23)
    _check_bf16(y, ref, "y", extra=size * ref.abs().amax() * 2.0 ** -20)
    _check_codes(c, s, ref, "codes")
    kept = ocq.add_rmsnorm(x, w, 1e-5, residual=res, residual_out=x)      # in place: what it reads it also writes
    assert kept[0] is x and torch.equal(x, r)
    assert torch.equal(kept[2].view(torch.uint8), c.view(torch.uint8)) and torch.equal(kept[3], s)


# ---------------------------------------------------------------- E4M3 segments that fill the GPU: longest first

@pytest.mark.parametrize("dim,n,requests,kv_heads", [(128, 13, 64, 8), (128, 13, 33, 8), (64, 13, 64, 8), (256, 13, 40, 8),
                                                     (128, 1, 64, 8), (128, 7, 50, 8), (128, 13, 9, 32)])
def test_attention_of_more_e4m3_segments_than_half_the_workgroups(dim, n, requests, kv_heads):
    """Uneven contexts (ties, empty ones, requests without new tokens, one far longer than the rest), all cut by the
    batch's own lengths; twice, so that the counts of the first call are seen by the second."""
    rng = np.random.default_rng(dim + n + requests)
    news = [n if i % 11 else 0 for i in range(requests)]
    kvs = [m + int(x) for m, x in zip(news, rng.integers(0, 700, requests))]
    kvs[0], kvs[3], kvs[4], kvs[7] = 0, 6000, kvs[5], 0
    news[3] = news[7] = n
    g = _gen(requests + n)
    batch, pages = make_batch(news, kvs, 32, g)
    cache = make_cache(pages, kv_heads, 32, dim, True, g)
    q = _bf((sum(news), 4 * kv_heads, dim), g)
    out, lse = check_attention(q, cache, batch, news, kvs)
    assert not batch.counters.any()
    again = ocq.paged_attention(q, cache, batch, want_lse=True)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


# ---------------------------------------------------------------- one append of many tokens, many of one

@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 64, True), (256, 256, False)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append_of_many_tokens_is_many_of_one(dim, rot, interleaved, e4m3):
    """The same rows of q, k and v give the same bits: q, the cache and its scales."""
    g, n, page = _gen(61), 13, 16
    lens = [37, 0, 50]
    whole, pages = make_batch([n] * 3, [l + n for l in lens], page, g)
    a = make_cache(pages, 2, page, dim, e4m3, g)
    b = ocq.PagedKVCache(*(None if x is None else x.clone() for x in (a.k, a.v, a.k_scale, a.v_scale)))
    rope = ocq.Rope.make(rot, interleaved, DEV, scaling="ntk", factor=4.0)
    q, k, v = _bf((3 * n, 4, dim), g), _bf((3 * n, 2, dim), g), _bf((3 * n, 2, dim), g)
    out = ocq.rope_append(q, k, v, rope, a, whole)
    start = torch.arange(4, dtype=torch.int32, device=DEV)
    for i in range(n):
        rows = torch.arange(i, 3 * n, n, device=DEV)
        one = ocq.TokenBatch(start, torch.tensor([l + i + 1 for l in lens], dtype=torch.int32, device=DEV),
                             whole.page_table, 1, 64)
        assert torch.equal(ocq.rope_append(q[rows], k[rows], v[rows], rope, b, one), out[rows])
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ---------------------------------------------------------------- the layer's MLP half

@pytest.mark.parametrize("prec_mode", [ocq.PREC_FP8, ocq.PREC_FP4])
def test_the_layer_is_its_operators_and_the_block(prec_mode):
    """The layer gives to the bit what the entry points give one by one; on that way the norm in front of the block is
    within its bounds of the 64-bit one, and the block within its own of the oracle's."""
    hidden, inter, n, seed = 256, 512, 50, 9
    layer, twin = (random_layer(hidden, inter, 8, 2, 64, 4, 16, seed=seed, device=DEV, prec_mode=prec_mode)
                   for _ in range(2))
    gen = _gen(9)
    batch = batch_of([n], [n], torch.arange(4, dtype=torch.int32, device=DEV)[None], DEV)
    x, pending = _bf((n, hidden), gen), _bf((n, hidden), gen)
    got, mlp = layer(x, pending, batch)

    x0, h0, _, _ = ocq.add_rmsnorm(x, twin.norm_in, twin.eps, residual=pending, want_y=True, want_codes=False)
    q, k, v = (h0 @ twin.w_qkv).view(n, 12, 64).split([8, 2, 2], 1)
    o, _ = ocq.paged_attention(ocq.rope_append(q, k, v, twin.rope, twin.cache, batch), twin.cache, batch)
    step = o.flatten(1) @ twin.w_o
    x1, h, _, _ = ocq.add_rmsnorm(x0, twin.norm_mlp, twin.eps, residual=step, want_y=True, want_codes=False)
    y = ocq.mlp_forward(twin.mlp.blob, h, hidden, inter, prec_mode)
    assert torch.equal(got, x1) and torch.equal(mlp, y)
    assert torch.equal(layer.cache.k, twin.cache.k) and torch.equal(layer.cache.v, twin.cache.v)

    sums, ref = _norm_ref(x0, twin.norm_mlp, twin.eps, step)
    size = x0.double().abs() + step.double().abs()
    _check_bf16(x1, sums, "x", extra=size * 2.0 ** -23)
    _check_bf16(h, ref, "h", extra=size * ref.abs().amax() * 2.0 ** -20)
    rng = np.random.default_rng(seed)
    w = [rng.standard_normal(s, dtype=np.float32) * np.float32(0.02)
         for s in ((inter, hidden), (inter, hidden), (hidden, inter))]

    def bits(t):
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    check_y(bits(y), O.block_reference(bits(h), *w, prec_mode)["y"])
