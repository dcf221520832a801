"""Attention over NVFP4 caches at its ends: rows of q next to zero, scales and units that meet them.
References and tolerances are those of test_gpu_nvfp4_cache.py."""

import pytest
import torch

from test_gpu_layer import _bf, _gen, make_batch
from test_gpu_nvfp4_cache import check_attention, make_cache

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
