"""The binding's handles of the operators around the block, what runs without a GPU: the numbers that they hand to the C
ABI, taken from CPU tensors (nothing is launched)."""

import pytest
import torch

from quantized_memory_bound_amd import ocq


@pytest.fixture
def cpu_handles(monkeypatch):
    """Handles accept CPU tensors, as if those were on the current device."""
    monkeypatch.setattr(ocq, "_gpu", lambda t, name: 0)


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
