"""The binding's handles of the operators around the block, what runs without a GPU: the numbers that they hand to the C
ABI, taken from CPU tensors (nothing is launched)."""

import ctypes

import pytest
import torch

from quantized_memory_bound_amd import ocq


@pytest.fixture
def cpu_handles(monkeypatch):
    """Handles accept CPU tensors, as if those were on the current device."""
    monkeypatch.setattr(ocq, "_gpu", lambda t, name: t.get_device())     # -1
    monkeypatch.setattr(ocq, "_torch", torch)
    monkeypatch.setattr(ocq, "_raw_stream", lambda i: 11)


def _ints(*shape):
    return torch.arange(int(torch.tensor(shape).prod()), dtype=torch.int32).reshape(shape)


def _batch(table):
    requests = len(table)
    return ocq.TokenBatch(torch.arange(requests + 1, dtype=torch.int32), torch.ones(requests, dtype=torch.int32), table,
                          1, 64)


# ---------------------------------------------------------------- page tables

@pytest.mark.parametrize("table", [
    _ints(7).expand(4, -1),                                 # one row for all requests
    _ints(64).as_strided((4, 7), (6, 1)),                   # rows that overlap
    _ints(64).as_strided((2, 7), (1, 1))])
def test_page_tables_whose_rows_share_entries_are_refused(cpu_handles, table):
    """Row r would be read at r * max_pages entries, past the tensor."""
    with pytest.raises(ocq.OcqError) as e:
        _batch(table)
    assert e.value.status == ocq.ERR_INVALID_ARG
    assert _batch(table.contiguous()).struct.table_stride == 7


@pytest.mark.parametrize("table,stride", [
    (_ints(4, 7), 7), (_ints(4, 12)[:, 2:9], 12), (_ints(8, 7)[::2], 14), (_ints(4, 1), 1), (_ints(4, 3)[:, 1:2], 3),
    (_ints(1, 7), 7), (_ints(7).expand(1, -1), 7), (_ints(64).as_strided((1, 7), (0, 1)), 7)])
def test_page_table_stride_is_the_tensors_own(cpu_handles, table, stride):
    """The last entry that a call may read lies in the tensor's storage."""
    b = _batch(table)
    assert b.struct.table_stride == stride and b.struct.max_pages == table.shape[1]
    last = table.storage_offset() + (len(table) - 1) * stride + table.shape[1] - 1
    assert last < table.untyped_storage().nbytes() // 4


# ---------------------------------------------------------------- counters of attention calls

class _Streams:
    """Stand-ins for torch.cuda's streams and for the library: which counters a call gets, and in whose order tensors
    were zeroed."""

    def __init__(self, monkeypatch):
        self.now, self.capturing, self.zeroed_on, self.calls = [11], set(), {}, []
        zeros = torch.zeros

        def spied(*a, **kw):
            t = zeros(*a, **kw)
            self.zeroed_on[t.data_ptr()] = self.now[-1]
            return t

        class _On:
            def __init__(this, handle):
                this.handle = handle

            def __enter__(this):
                self.now.append(this.handle)

            def __exit__(this, *a):
                self.now.pop()
        monkeypatch.setattr(torch, "zeros", spied)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
        monkeypatch.setattr(torch.cuda, "stream", _On)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.now[-1] in self.capturing)
        monkeypatch.setattr(ocq, "_raw_stream", lambda i: self.now[-1])
        monkeypatch.setattr(ocq, "_empty", lambda shape, dtype, index, stream: torch.empty(shape, dtype=dtype))
        monkeypatch.setattr(ocq, "lib", lambda: self)

    def ocq_attention_workspace_bytes(self, *a):
        return 0

    def ocq_paged_attention(self, *a):
        batch = ctypes.cast(a[5], ctypes.POINTER(ocq.TokenBatchStruct)).contents
        self.calls.append((batch.counters_dev, a[-1]))
        return 0


def test_attention_calls_count_in_memory_of_their_own_stream(cpu_handles, monkeypatch):
    streams = _Streams(monkeypatch)
    cache = ocq.PagedKVCache(*(torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    batch, q = _batch(_ints(2, 2)), torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    home = batch.counters.data_ptr()
    for stream in (None, 22, 22, None, 33, 22):
        ocq.paged_attention(q, cache, batch, stream=stream)
    assert [h for _, h in streams.calls] == [11, 22, 22, 11, 33, 22]
    for counters, handle in streams.calls:
        assert streams.zeroed_on[counters] == handle
    assert len({c for c, _ in streams.calls}) == 3
    assert {t.data_ptr() for t in batch.counters_of.values()} == {c for c, _ in streams.calls}   # kept with the batch
    # captured calls add no fill to the graph; afterwards the same stream has counters of its own
    streams.calls.clear()
    streams.capturing = {44}
    for _ in range(2):
        ocq.paged_attention(q, cache, batch, stream=44)
    assert [c for c, _ in streams.calls] == [home, home]
    streams.capturing = set()
    ocq.paged_attention(q, cache, batch, stream=44)
    assert streams.calls[-1][0] not in (home, None) and streams.zeroed_on[streams.calls[-1][0]] == 44
    streams.now[0] = 55                                    # the current stream is another one
    ocq.paged_attention(q, cache, batch)
    assert streams.zeroed_on[streams.calls[-1][0]] == 55


# ---------------------------------------------------------------- sizes of launches

@pytest.mark.parametrize("requests,tokens,max_new,heads,kv_heads", [
    (65536, 65536 + 8192, 8192, 8, 8),           # 2^25 workgroups of 256 lanes
    (4096, 4095 + 32768, 32768, 32, 8),          # one long chunk among many requests
    (65536, 1 << 17, 1, 4096, 4096)])            # one token each, many heads
def test_attention_refuses_more_lanes_than_a_launch_holds(requests, tokens, max_new, heads, kv_heads):
    p = 4096                                     # an aligned address that no refused call reads
    cache = ocq.KVCacheStruct(k_dev=p, v_dev=p, page_stride=kv_heads * 16 * 64, head_stride=16 * 64, token_stride=64,
                              num_pages=4, page_size=16, kv_heads=kv_heads, head_dim=64, format=0)
    batch = ocq.TokenBatchStruct(q_start_dev=p, kv_lens_dev=p, page_table_dev=p, table_stride=4, requests=requests,
                                 tokens=tokens, max_pages=4, max_new=max_new, max_kv=60, counters_dev=p)
    status = ocq.lib().ocq_paged_attention(p, heads * 64, 64, heads, ctypes.byref(cache), ctypes.byref(batch), 0.125, 0,
                                           0, p, None, p, 1 << 50, None)
    assert status == ocq.ERR_UNSUPPORTED and "launch" in ocq.last_error()


def _e4m3(scale_token_stride, page_size):
    p = 4096                                     # an aligned address that no refused call reads
    return ocq.KVCacheStruct(k_dev=p, v_dev=p, k_scale_dev=p, v_scale_dev=p, page_stride=2 * page_size * 64,
                             head_stride=page_size * 64, token_stride=64, scale_page_stride=8, scale_head_stride=4,
                             scale_token_stride=scale_token_stride, num_pages=4, page_size=page_size, kv_heads=2,
                             head_dim=64, format=1)


@pytest.mark.parametrize("step,page_size,status", [(1 << 26, 32, ocq.ERR_UNSUPPORTED), (1 << 25, 64, ocq.ERR_UNSUPPORTED),
                                                   (1 << 30, 2, ocq.ERR_UNSUPPORTED), (1 << 25, 32, ocq.OK),
                                                   ((1 << 30) - 1, 2, ocq.OK), (1 << 40, 1, ocq.OK)])
def test_scales_whose_offsets_pass_32_bits_of_bytes_are_refused(step, page_size, status):
    """Attention would read another row's scale.  (No tokens: an accepted cache has nothing to do.)"""
    batch = ocq.TokenBatchStruct(requests=0, tokens=0)
    cache = _e4m3(step, page_size)
    assert ocq.lib().ocq_paged_attention(None, 64, 64, 4, ctypes.byref(cache), ctypes.byref(batch), 0.125, 0, 0, None,
                                         None, None, 0, None) == status
    assert ocq.lib().ocq_rope_append(None, 64, 64, None, 64, 64, None, 64, 64, 4, None, 64, 0, 1.0, None,
                                     ctypes.byref(cache), ctypes.byref(batch), None, None) == status


# ---------------------------------------------------------------- numbers beyond 32 bits

BEYOND = [1 << 31, (1 << 32) + 5, -(1 << 32) + 5]


@pytest.mark.parametrize("value", BEYOND)
def test_numbers_beyond_32_bits_are_refused(cpu_handles, monkeypatch, value):
    """ctypes would pass their low 32 bits: a window of 2^32 + 5 would be one of 5."""
    cache = ocq.PagedKVCache(*(torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    batch, q = _batch(_ints(2, 2)), torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    batch.of(2)
    _Streams(monkeypatch)
    ints = torch.arange(3, dtype=torch.int32), torch.ones(2, dtype=torch.int32), _ints(2, 2)
    for call in (lambda: ocq.paged_attention(q, cache, batch, window=value),
                 lambda: ocq.paged_attention(q, cache, batch, window=8, sinks=value),
                 lambda: ocq.attention_workspace_bytes(1, cache, batch, value),
                 lambda: ocq.TokenBatch(*ints, value, 64), lambda: ocq.TokenBatch(*ints, 1, value),
                 lambda: ocq.TokenBatch(*ints, 1, 64, tokens=value)):
        with pytest.raises(ocq.OcqError) as e:
            call()
        assert e.value.status == ocq.ERR_INVALID_ARG


def test_tensors_of_more_rows_than_32_bits_are_refused(cpu_handles):
    row = torch.zeros(1, 8, dtype=torch.bfloat16)
    with pytest.raises(ocq.OcqError) as e:
        ocq.add_rmsnorm(row.expand((1 << 32) + 3, 8), row[0])
    assert e.value.status == ocq.ERR_INVALID_ARG
    page = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16).expand((1 << 32) + 3, 1, 16, 64)
    with pytest.raises(ocq.OcqError) as e:
        ocq.PagedKVCache(page, page)
    assert e.value.status == ocq.ERR_INVALID_ARG
