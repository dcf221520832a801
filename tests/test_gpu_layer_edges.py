"""The operators around the block where their inputs leave the ordinary range: values that are not finite or next to
zero, and the launches' largest sizes.  Tolerances as in test_gpu_layer.py."""

import pytest
import torch

from quantized_memory_bound_amd import ocq
from test_gpu_layer import DEV, E4M3, _bf, _check_codes, _gen, check_attention, make_batch, make_cache

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


# ---------------------------------------------------------------- rows next to zero

TINY = [2.0 ** -110, 2.0 ** -119, 2.0 ** -121, 2.0 ** -124, 2.0 ** -126]


def _check_tiny(codes, scales, ref, what):
    """Scales below 2^-126 are rounded to a multiple of 2^-149; each code is the nearest to the quotient by its own
    scale: half a step of 2^-4 relative or 2^-10 (subnormal), and the largest may be clipped by the scale's rounding."""
    ref = ref.double()
    s, got = scales.double(), codes.view(E4M3).double() * scales.double()[..., None]
    exact = ref.abs().amax(-1) / 448
    assert torch.all((s - exact).abs() <= exact * 2.0 ** -20 + 2.0 ** -149), what
    tol = ref.abs() * (2.0 ** -4 + 2.0 ** -18) + s[..., None] * (2.0 ** -10 + 2.0 ** -18) + 448 * 2.0 ** -149
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), "%s: %d of %d codes off" % (what, int(bad.sum()), bad.numel())


@pytest.mark.parametrize("size", TINY)
def test_append_of_tiny_values(size):
    """The scale of a head may be so small that its reciprocal overflows."""
    g = _gen(21)
    batch, pages = make_batch([13], [40], 16, g)
    cache = make_cache(pages, 2, 16, 128, True, g)
    k, v = ((_bf((13, 2, 128), g).clamp(-4, 4).float() * size).to(torch.bfloat16) for _ in range(2))
    k[3, 0, 1:] = v[3, 0, 1:] = 0
    zero = torch.zeros(13, dtype=torch.int32, device=DEV)                 # position 0: nothing is turned
    ocq.rope_append(_bf((13, 4, 128), g), k, v, ocq.Rope.make(128, device=DEV), cache, batch, positions=zero)
    ids, rows = _slots(batch, cache, 0, torch.arange(27, 40, device=DEV))
    _check_tiny(cache.k[ids, :, rows], cache.k_scale[ids, :, rows], k, "k")
    _check_tiny(cache.v[ids, :, rows], cache.v_scale[ids, :, rows], v, "v")


@pytest.mark.parametrize("size", TINY)
@pytest.mark.parametrize("hidden", [512, 2048, 16384, 65536])
def test_norm_to_tiny_values(size, hidden):
    g = _gen(22)
    x, w = _bf((3, hidden), g).clamp(-4, 4), (_bf((hidden,), g).clamp(-2, 2).float() * size).to(torch.bfloat16)
    x[:, ::5] = 0
    _, _, c, s = ocq.add_rmsnorm(x, w, 0.0)
    h = x.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True)) * w.double()
    # y itself is rounded to a multiple of 2^-149 below 2^-126
    err = 2.0 ** -149
    assert torch.all((s.double() - y.abs().amax(-1) / 448).abs() <= s.double() * 2.0 ** -20 + 2 * err)
    got = c.view(E4M3).double() * s.double()[:, None]
    tol = y.abs() * (2.0 ** -4 + 2.0 ** -18) + s.double()[:, None] * (2.0 ** -10 + 2.0 ** -18) + 450 * err
    assert torch.all((got - y).abs() <= tol)


# ---------------------------------------------------------------- streams

def test_attention_on_a_stream_that_the_batch_was_not_made_on():
    """The batch is made on a stream that is still busy, in memory that holds other numbers, and dropped while its call
    is waiting: neither reaches the call's counts."""
    g = _gen(31)
    news, kvs = [13, 13], [3000, 2000]
    first, pages = make_batch(news, kvs, 32, g)
    cache, q = make_cache(pages, 2, 32, 128, False, g), _bf((26, 8, 128), g)
    want, lse = check_attention(q, cache, first, news, kvs)
    home, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(home):
            spoiled = [torch.full((ocq.ATTENTION_COUNTERS,), 7, dtype=torch.int32, device=DEV) for _ in range(4)]
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)                        # about 10 ms
            del spoiled
            batch = ocq.TokenBatch(first.q_start, first.kv_lens, first.page_table, 13, 3000)
        out = ocq.paged_attention(q, cache, batch, want_lse=True, stream=side)
        side.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], lse)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = ocq.paged_attention(q, cache, batch, want_lse=True, stream=side)
        del batch
        with torch.cuda.stream(home):
            again = [torch.full((ocq.ATTENTION_COUNTERS,), 7, dtype=torch.int32, device=DEV) for _ in range(8)]
        torch.cuda.synchronize()                                 # home's fills too, read on another stream below
        assert torch.equal(out[0], want) and torch.equal(out[1], lse)
        assert all(bool((t == 7).all()) for t in again)


def test_one_batch_on_several_streams_and_in_a_graph():
    g = _gen(32)
    news, kvs = [5, 5], [2000, 900]
    batch, pages = make_batch(news, kvs, 64, g)
    cache, q = make_cache(pages, 2, 64, 128, True, g), _bf((10, 8, 128), g)
    want, lse = check_attention(q, cache, batch, news, kvs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ocq.paged_attention(q, cache, batch, want_lse=True)
    sides = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        outs = [ocq.paged_attention(q, cache, batch, want_lse=True, stream=s) for s in sides]   # at the same time
        captured[0].zero_()
        graph.replay()
        outs += [ocq.paged_attention(q, cache, batch, want_lse=True), captured]
        torch.cuda.synchronize()
        for a, b in outs:
            assert torch.equal(a, want) and torch.equal(b, lse)
    assert not any(bool(c.any()) for c in batch.counters_of.values())


# ---------------------------------------------------------------- sizes of launches

def test_norm_of_its_most_rows():
    """2^24 rows of 256 lanes are 2^32 of them.  Rows overlap in memory (8 elements apart): all differ."""
    rows, hidden = 1 << 24, 520
    x = _bf((8 * (rows - 1) + hidden,), _gen(41)).as_strided((rows, hidden), (8, 1))
    w = _bf((hidden,), _gen(42))
    scales = torch.full((rows,), -1.0, device=DEV)
    codes = ocq.add_rmsnorm(x, w, 1e-6, scales=scales)[2]
    assert bool((scales > 0).all())
    some = torch.tensor([0, 1, 1 << 20, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, rows - 2, rows - 1], device=DEV)
    h = x[some].double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    _check_codes(codes[some], scales[some], y, "codes")


def test_append_of_more_tokens_than_one_launch_holds():
    tokens, page = (1 << 24) + 5, 1024
    g = _gen(43)
    q, k, v = (_bf((8 * (tokens - 1) + 64,), g).as_strided((tokens, 1, 64), (8, 64, 1)) for _ in range(3))
    pages = -(-tokens // page)
    cache = ocq.PagedKVCache.allocate(pages, page, 1, 64, device=DEV)
    table = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)[None]
    batch = ocq.TokenBatch(torch.tensor([0, tokens], dtype=torch.int32, device=DEV),
                           torch.tensor([tokens], dtype=torch.int32, device=DEV), table, tokens, tokens)
    zero = torch.zeros(tokens, dtype=torch.int32, device=DEV)          # position 0: nothing is turned
    out = ocq.rope_append(q, k, v, ocq.Rope.make(64, device=DEV), cache, batch, positions=zero)
    at = torch.arange(tokens, device=DEV)
    for part in at.split(1 << 20):
        ids, rows = table[0][part // page].long(), part % page
        assert torch.equal(out[part], q[part])
        assert torch.equal(cache.k[ids, 0, rows], k[part, 0]) and torch.equal(cache.v[ids, 0, rows], v[part, 0])


# ---------------------------------------------------------------- scales that lie far apart

def test_scales_of_one_page_as_far_apart_as_may_be():
    """31 times 2^25 elements are just within 2^30, their offsets in bytes within 2^32 and past 2^31."""
    g, page, step = _gen(51), 32, 1 << 25
    news, kvs = [13, 1, 40], [200, 90, 70]
    batch, pages = make_batch(news, kvs, page, g)
    room = torch.empty((page - 1) * step + 8 * pages, device=DEV)
    ks, vs = (room.as_strided((pages, 2, page), (8, 4, step), at) for at in (0, 2))
    plain = make_cache(pages, 2, page, 128, True, g)
    ks.copy_(plain.k_scale)
    vs.copy_(plain.v_scale)
    cache = ocq.PagedKVCache(plain.k, plain.v, ks, vs)
    q, k, v = _bf((54, 8, 128), g), _bf((54, 2, 128), g), _bf((54, 2, 128), g)
    q = ocq.rope_append(q, k, v, ocq.Rope.make(128, device=DEV), cache, batch)
    check_attention(q, cache, batch, news, kvs)                       # rows of many: 128-row tiles
    for r, (n, kv) in enumerate(zip(news[:2], kvs[:2])):              # up to 64 rows, up to 16
        one, _ = make_batch([n], [kv], page, g)
        one.page_table[0] = batch.page_table[r, : one.page_table.shape[1]]
        check_attention(q[13 * r: 13 * r + n], cache, one, [n], [kv])


# ---------------------------------------------------------------- no eps

@pytest.mark.parametrize("hidden", [72, 512, 2048, 4096, 8192, 16384, 32768, 65536])
def test_norm_without_eps_of_zero_rows_and_of_rows_whose_squares_vanish(hidden):
    """A zero row has scale 0 and codes 0 whatever its y (0 / 0) is; a row that is not zero but whose squares are 0 in
    fp32 has no norm: scale NaN, codes 0; the others are as ever."""
    g = _gen(hidden + 1)
    x, w = _bf((9, hidden), g), _bf((hidden,), g)
    w[w == 0] = 1
    x[[1, 6]] = 0
    x[3] = 0
    x[3, hidden // 2] = 1e-30
    x[4] = 1e-30
    _, _, c, s = ocq.add_rmsnorm(x, w, 0.0)
    assert (s[[1, 6]] == 0).all() and not c[[1, 6]].view(torch.uint8).any()
    assert torch.isnan(s[[3, 4]]).all() and not c[[3, 4]].view(torch.uint8).any()
    rest = [0, 2, 5, 7, 8]
    h = x[rest].double()
    _check_codes(c[rest], s[rest], h / torch.sqrt(h.square().mean(-1, keepdim=True)) * w.double(), "codes")
    s = ocq.add_rmsnorm(x, w, 1e-6)[3]
    assert (s[[1, 6]] == 0).all() and (s[[3, 4]] > 0).all()
