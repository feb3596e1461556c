"""CPU checks of the tree and cache entry points: the struct matches the header, workspace sizes cover the
partial results, and bad calls are refused on the host, before any launch (no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EWORKSPACE = 1, 8


@pytest.fixture(scope="module")
def ds():
    from dspark_draft_selection_gb300.build import LIB, build
    if not os.path.exists(LIB):
        build()
    import dspark_draft_selection_gb300 as ds
    return ds


def _cache(ds, **kw):
    v = dict(k=4096, v=8192, dtype=0, n_layers=1, layer_stride=0, page_stride=16 * 2 * 64, token_stride=128, head_stride=64,
             num_pages=10, page_size=16, heads=2, head_dim=64, page_table=256, ld_table=4, table_pages=4)
    v.update(kw)
    return ds._binding.KVCache(*(v[n] for n, _ in ds._binding.KVCache._fields_))


def test_the_cache_struct_has_the_headers_fields(ds):
    text = open(os.path.join(ROOT, "include", "dspark.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} dspark_kvcache;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for line in body.split(";") for n in re.sub(r"^\s*(const )?\w+", "", line).split(",") if n.strip(" *\n")]
    assert [n.strip() for n in names] == [n for n, _ in ds._binding.KVCache._fields_]


BAD_CACHES = [dict(k=None), dict(v=None), dict(page_table=None), dict(dtype=5), dict(k=4097), dict(page_stride=-1), dict(num_pages=0),
              dict(num_pages=2 ** 31), dict(page_size=0), dict(page_size=65537), dict(heads=0), dict(heads=1025), dict(head_dim=12),
              dict(head_dim=264), dict(head_dim=0), dict(ld_table=3), dict(table_pages=0)]


def test_refusals(ds):
    lib, f, ws = ds.lib(), ctypes.c_void_p(256), 1 << 28
    att = lambda c, q=f, ldq=256, R=1, T=2, Hq=4, ctx=f, scale=0.1, cap=0.0, out=f, ldo=256, w=f, wn=ws, st=f: lib.dspark_tree_attention(  # noqa: E731
        q, ldq, R, T, Hq, ctypes.byref(c) if c else None, ctx, None, None, scale, cap, out, ldo, None, w, wn, st, None)
    rope = lambda c, q=f, ldq=256, ldk=128, R=1, T=2, Hq=4, A=1, P=8, rot=64, out=f, ldo=256: lib.dspark_rope_append(  # noqa: E731
        q, ldq, f, ldk, f, 128, R, T, Hq, f, A, f, P, rot, None, 0, ctypes.byref(c) if c else None, f, None, out, ldo, f, None)
    commit = lambda c, R=1, T=2, new=ctypes.c_void_p(512): lib.dspark_cache_commit(  # noqa: E731
        ctypes.byref(c) if c else None, f, f, f, R, T, new, f, None)
    good = _cache(ds)
    for bad in BAD_CACHES:
        c = _cache(ds, **bad)
        assert att(c) == EINVAL and rope(c) == EINVAL and commit(c) == EINVAL, bad
    assert att(None) == EINVAL and rope(None) == EINVAL and commit(None) == EINVAL
    assert commit(_cache(ds, n_layers=0)) == EINVAL and commit(_cache(ds, layer_stride=-1)) == EINVAL
    for kw in (dict(q=None), dict(ldq=255), dict(R=-1), dict(R=1025), dict(T=0), dict(T=513), dict(Hq=3), dict(Hq=0), dict(ctx=None),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")),
               dict(out=None), dict(ldo=255), dict(st=None), dict(q=ctypes.c_void_p(257))):
        assert att(good, **kw) == EINVAL, kw
    for kw in (dict(w=None), dict(wn=100), dict(w=ctypes.c_void_p(260))):
        assert att(good, **kw) == EWORKSPACE, kw
    for kw in (dict(q=None), dict(ldq=200), dict(ldk=100), dict(T=0), dict(Hq=5), dict(A=0), dict(A=9), dict(P=0), dict(rot=0),
               dict(rot=3), dict(rot=66), dict(out=None), dict(ldo=200), dict(ldo=512, out=f), dict(R=2 ** 31, T=2)):
        assert rope(good, **kw) == EINVAL, kw
    for kw in (dict(R=65536), dict(T=0), dict(T=513), dict(new=None), dict(new=f)):
        assert commit(good, **kw) == EINVAL, kw
    for n in (0, 513):
        assert lib.dspark_tree_mask(f, None, None, 1, n, f, f, f, None) == EINVAL
        assert lib.dspark_tree_accept(f, None, f, None, 1, n, f, f, f, f, None) == EINVAL
    assert lib.dspark_tree_mask(f, None, None, 1, 4, None, f, f, None) == EINVAL
    assert lib.dspark_tree_accept(None, None, f, None, 1, 4, f, f, f, f, None) == EINVAL


def test_empty_batches_launch_nothing(ds):
    lib, c = ds.lib(), ctypes.byref(_cache(ds))
    assert lib.dspark_tree_mask(None, None, None, 0, 4, None, None, None, None) == 0
    assert lib.dspark_tree_accept(None, None, None, None, 0, 4, None, None, None, None, None) == 0
    assert lib.dspark_rope_append(None, 256, None, 128, None, 128, 0, 2, 4, None, 1, None, 8, 64, None, 0, c, None, None, None, 256,
                                  None, None) == 0
    assert lib.dspark_tree_attention(None, 256, 0, 2, 4, c, None, None, None, 0.1, 0.0, None, 256, None, None, 0, None, None) == 0
    assert lib.dspark_cache_commit(c, None, None, None, 0, 2, None, None, None) == 0


def test_workspace_covers_two_partial_results_per_block(ds):
    for T, Hq, H, D in ((1, 8, 8, 8), (64, 32, 4, 128), (512, 64, 1, 256), (13, 12, 4, 80)):
        n = ds.dspark_workspace_size(ds.OP_TREE_ATTENTION, 3, T, Hq * D, H)
        rows = T * Hq // H
        assert n >= 2 * 148 * min(rows, 256) * (D * 4 + 8) and n >= 4 * 148 * min(rows, 64) * (D * 4 + 8)
    assert ds.dspark_workspace_size(ds.OP_TREE_ATTENTION, 0, 4, 256, 2) == 0
