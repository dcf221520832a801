"""The operators around the block where their inputs leave the ordinary range: values that are not finite or next to
zero, and the launches' largest sizes.  Tolerances as in test_gpu_layer.py."""

import pytest
import torch

from quantized_memory_bound_amd import ocq
from test_gpu_layer import DEV, E4M3, _bf, _check_codes, _gen, make_batch, make_cache

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- append to an E4M3 cache

def _slots(batch, cache, r, places):
    return batch.page_table[r][places // cache.page_size].long(), places % cache.page_size


@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 48), (256, 256)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_append_of_values_that_are_not_finite(dim, rot, which):
    """One NaN, a head of NaN, and infinities: the head's scale is NaN and its codes 0, every other head is as ever, and
    attention gives NaN to the tokens that see the row."""
    g = _gen(dim)
    n, kv, page = 13, 90, 16
    batch, pages = make_batch([n], [kv], page, g)
    cache = make_cache(pages, 2, page, dim, True, g)
    rope = ocq.Rope.make(rot, device=DEV)
    q, k, v = _bf((n, 4, dim), g), _bf((n, 2, dim), g), _bf((n, 2, dim), g)
    x = k if which == "k" else v
    nan, inf = float("nan"), float("inf")
    x[4, 0, dim - 1], x[5, 1], x[7, 0, 3], x[9, 1, 8] = nan, nan, inf, -inf
    bad = torch.zeros((n, 2), dtype=torch.bool, device=DEV)
    bad[[4, 5, 7, 9], [0, 1, 0, 1]] = True
    clean_k = ocq.rope_append(k, k, v, rope, make_cache(pages, 2, page, dim, False, g), batch)   # rotated k in bf16
    q = ocq.rope_append(q, k, v, rope, cache, batch)
    ids, rows = _slots(batch, cache, 0, torch.arange(kv - n, kv, device=DEV))
    pools = dict(k=(cache.k, cache.k_scale), v=(cache.v, cache.v_scale))
    for name, (codes, scales) in pools.items():
        c, s = codes[ids, :, rows], scales[ids, :, rows]
        hit = bad if name == which else torch.zeros_like(bad)
        assert torch.equal(torch.isnan(s), hit)
        assert not c.view(torch.uint8)[hit].any()
        if name == "v":
            _check_codes(c[~hit], s[~hit], v.double()[~hit], "v")
        else:   # against the bf16 rounding of the same rotated values: 2^-8 of each besides
            got, want = c[~hit].view(E4M3).double() * s[~hit].double()[..., None], clean_k.double()[~hit]
            top = want.abs().amax(-1, keepdim=True)
            assert torch.all((got - want).abs() <= want.abs() * (2.0 ** -4 + 2.0 ** -7) + top * 2.0 ** -18)
    out, lse = ocq.paged_attention(q, cache, batch, want_lse=True)
    sees = bad.cumsum(0).bool().repeat_interleave(2, 1)      # [n, heads]: a bad row at or before the token
    assert torch.isnan(out[sees].float()).all()
    if which == "k":
        assert torch.isnan(lse[sees]).all() and torch.isfinite(out[~sees].float()).all()


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("hidden", [72, 2048, 4096, 8192, 16384, 32768, 65536])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_norm_with_a_weight_that_is_not_finite(hidden, value):
    """Every row's y is not finite in that place: scale NaN, codes 0; where the row is 0 there (0 x inf) as well."""
    g = _gen(hidden)
    x, w = _bf((5, hidden), g), _bf((hidden,), g)
    w[hidden - 3] = value
    x[2, hidden - 3] = 0
    _, y, c, s = ocq.add_rmsnorm(x, w, 1e-6, want_y=True)
    assert torch.isnan(s).all() and not c.view(torch.uint8).any()
    got = y.float().isfinite()
    assert not got[:, hidden - 3].any() and got[:, : hidden - 3].all() and got[:, hidden - 2:].all()
    w[hidden - 3] = 1
    s = ocq.add_rmsnorm(x, w, 1e-6)[3]
    assert torch.isfinite(s).all()
