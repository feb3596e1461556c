"""Where a commit may write the new lengths: the blocks of a request's layers, keys and values read its committed length, its count and its
path while one of them writes the new length, so no array of those may share memory with it. Refused on the host, before any launch."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = 1
CALLS = ["dspark_cache_commit_q8", "dspark_cache_commit"]


@pytest.fixture(scope="module")
def ds():
    from dspark_draft_selection_gb300.build import LIB, build
    if not os.path.exists(LIB):
        build()
    import dspark_draft_selection_gb300 as ds
    return ds


def _cache(ds, call):
    v = dict(k=4096, v=8192, k_scale=512, v_scale=768, code=0, dtype=0, n_layers=2, layer_stride=0, page_stride=16 * 2 * 64, token_stride=128,
             head_stride=64, scale_layer_stride=0, scale_page_stride=64, scale_token_stride=2, scale_head_stride=32, num_pages=10,
             page_size=16, heads=2, head_dim=64, page_table=256, ld_table=4, table_pages=4)
    kind = ds._binding.QCache if call.endswith("_q8") else ds._binding.KVCache
    return kind(*(v[n] for n, _ in kind._fields_))


# R = 4, T = 3: lengths and counts of 16 bytes, a path of 48
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("ctx,acc,path,new", [(1024, 2048, 4096, 2048), (1024, 2048, 4096, 2044), (1024, 2048, 4096, 2060), (1024, 2048, 4096, 4096),
                                              (1024, 2048, 4096, 4140), (1024, 2048, 4096, 4084), (1024, 2048, 4096, 1024), (1024, 2048, 4096, 1036),
                                              (1024, 2048, 4096, 1012), (1024, 2048, None, 2052), (1024, 2048, None, 2040), (1024, 2048, None, 1024),
                                              (1024, 2048, None, 1028)])
def test_lengths_among_what_is_read_are_refused(ds, call, ctx, acc, path, new):
    cache = ctypes.byref(_cache(ds, call))
    assert getattr(ds.lib(), call)(cache, ctx, path, acc, 4, 3, new, 256, None) == EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_lengths_that_are_not(ds, call):
    """Right behind and right before each array, and, without a path, the counts themselves."""
    layers, R, T, H, D, page = 2, 4, 3, 2, 64, 16
    cache = ds.q8_cache(8, page, H, D, layers=layers) if call.endswith("_q8") else \
        tuple(torch.zeros((layers, 8, page, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda").reshape(R, 2)
    commit = lambda *a, **kw: getattr(ds, call)(*((cache,) if call.endswith("_q8") else cache), table, *a, **kw)  # noqa: E731
    pool = torch.zeros(6 * R + R * T, dtype=torch.int32, device="cuda")
    ctx, acc, path = pool[R:2 * R], pool[3 * R:4 * R], pool[5 * R:5 * R + R * T].view(R, T)
    ctx.copy_(torch.tensor([5, 0, 17, 20]))
    acc.copy_(torch.tensor([1, 0, -1, 2]))
    path.copy_(torch.tensor([[0, 2, -1], [0, -1, -1], [-1, -1, -1], [0, 1, 2]]))
    want = [7, 1, 17, 23]
    for at in (0, 2 * R, 4 * R, 5 * R + R * T):
        new, status = commit(ctx, path, acc, out=pool[at:at + R])
        assert new.tolist() == want and ds.read_status(status) == 0
    for bad in (acc, path.view(-1)[:R], pool[3 * R - 1:4 * R - 1], pool[3 * R + 1:4 * R + 1], pool[R - 1:2 * R - 1]):
        with pytest.raises(ds.DsparkError):
            commit(ctx, path, acc, out=bad)
    new, status = commit(ctx, None, acc, T=T, out=acc)
    assert acc.tolist() == want and ds.read_status(status) == 0
