"""CPU checks of what the binding makes of the tree operators' tensors (no GPU needed: tensors of the host get as far as the
check that they are the device's)."""
import pytest
import torch

import dspark_draft_selection_gb300 as ds

R, T, H, D, PAGE = 3, 2, 2, 64, 16


def _calls(table):
    """The three calls that take a page table, with everything else as it should be."""
    k = torch.zeros((8, PAGE, H, D), dtype=torch.bfloat16)
    q, n = torch.zeros((table.shape[0], T, H, D), dtype=torch.bfloat16), torch.zeros(table.shape[0], dtype=torch.int32)
    pos, path = (torch.zeros((table.shape[0], T), dtype=torch.int32) for _ in range(2))
    return (lambda: ds.dspark_rope_append(q, q, q, pos, torch.zeros(4, D), k, k, table, n),
            lambda: ds.dspark_tree_attention(q, k, k, table, n),
            lambda: ds.dspark_cache_commit(k, k, table, n, path, n))


@pytest.mark.parametrize("table", [torch.arange(4).int()[None].expand(R, 4),                  # one row for all requests
                                   torch.arange(8).int().as_strided((R, 4), (2, 1))])         # rows that overlap
def test_tables_whose_rows_overlap_are_refused(table):
    for call in _calls(table):
        with pytest.raises(ValueError, match="rows overlap"):
            call()


@pytest.mark.parametrize("table,ld", [(torch.zeros((R, 4), dtype=torch.int32), 4), (torch.zeros((R, 9), dtype=torch.int32)[:, :4], 9),
                                      (torch.zeros((R, 2, 4), dtype=torch.int32)[:, 1], 8),
                                      (torch.zeros((1, 9), dtype=torch.int32)[:, :4], 4),     # one row: any stride
                                      (torch.zeros(4, dtype=torch.int32).expand(1, 4), 4),
                                      (torch.zeros(4, dtype=torch.int32).as_strided((1, 4), (0, 1)), 4),
                                      (torch.zeros((0, 4), dtype=torch.int32), 4)])
def test_the_tables_row_stride_is_passed_on(table, ld, monkeypatch):
    monkeypatch.setattr(ds._binding, "_p", lambda t: t.data_ptr() or 16)
    k = torch.zeros((8, PAGE, H, D), dtype=torch.bfloat16)
    packed, heads, cols, requests = ds._binding._kvcache(k, k, table)
    c = ds._binding.KVCache.from_buffer_copy(packed)
    assert (c.ld_table, c.table_pages, requests, heads, cols) == (ld, 4, table.shape[0], H, D)
    assert [getattr(c, f) for f in ("page_stride", "token_stride", "head_stride", "num_pages", "page_size")] == [PAGE * H * D, H * D, D, 8, PAGE]
    for call in _calls(table) if table.shape[0] else ():
        with pytest.raises(Exception) as e:                  # past the table's check, to the one of the device
            monkeypatch.undo()
            call()
        assert "device tensors" in str(e.value)


class _Stream:
    cuda_stream = 77


@pytest.mark.parametrize("has", [(), ("_cuda_getDevice",), ("_cuda_getCurrentRawStream",)])
def test_the_current_stream_without_torchs_own_functions(has, monkeypatch):
    """A torch without both of them: the public call gives the handle."""
    raw, device = ds._binding._stream_calls(type("C", (), {f: staticmethod(lambda *_: 3) for f in has}))
    monkeypatch.setattr(ds._binding, "_raw_stream", raw)
    monkeypatch.setattr(ds._binding, "_device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: _Stream())
    assert ds._binding._stream(None) == 77
    other = _Stream()
    other.cuda_stream = 5
    assert ds._binding._stream(other) == 5


@pytest.mark.gpu
def test_the_current_streams_handle():
    side = torch.cuda.Stream()
    assert ds._binding._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert ds._binding._stream(None) == side.cuda_stream
