"""CPU checks of the entry points of the cache in 8 bits and of dspark_tree_verify: the struct matches the header, bad calls are
refused on the host before any launch, and the binding refuses tensors that do not fit (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

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
    v = dict(k=4096, v=8192, k_scale=512, v_scale=768, code=0, n_layers=1, layer_stride=0, page_stride=16 * 2 * 64, token_stride=128,
             head_stride=64, scale_layer_stride=0, scale_page_stride=64, scale_token_stride=2, scale_head_stride=32, num_pages=10,
             page_size=16, heads=2, head_dim=64, page_table=256, ld_table=4, table_pages=4)
    v.update(kw)
    return ds._binding.QCache(*(v[n] for n, _ in ds._binding.QCache._fields_))


def test_the_cache_struct_has_the_headers_fields(ds):
    text = open(os.path.join(ROOT, "include", "dspark.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} dspark_qcache;", text).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for line in body.split(";") for n in re.sub(r"^\s*(const )?\w+", "", line).split(",") if n.strip(" *\n")]
    assert [n.strip() for n in names] == [n for n, _ in ds._binding.QCache._fields_]


BAD_CACHES = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(page_table=None), dict(code=2), dict(code=-1),
              dict(page_stride=-1), dict(scale_page_stride=-1), dict(scale_token_stride=-1), dict(scale_head_stride=-1), dict(num_pages=0),
              dict(num_pages=2 ** 31), dict(page_size=0), dict(page_size=65537), dict(heads=0), dict(heads=1025), dict(head_dim=12),
              dict(head_dim=264), dict(head_dim=0), dict(ld_table=3), dict(table_pages=0)]


def test_refusals(ds):
    lib, f, ws = ds.lib(), ctypes.c_void_p(256), 1 << 28
    g = ctypes.c_void_p(512)
    ref = lambda c: ctypes.byref(c) if c else None  # noqa: E731
    att = lambda c, q=f, ldq=256, dt=0, R=1, T=2, Hq=4, ctx=f, scale=0.1, cap=0.0, out=f, ldo=256, w=f, wn=ws, st=f: lib.dspark_tree_attention_q8(  # noqa: E731
        q, ldq, dt, R, T, Hq, ref(c), ctx, None, None, scale, cap, out, ldo, None, w, wn, st, None)
    rope = lambda c, q=f, ldq=256, ldk=128, dt=0, R=1, T=2, Hq=4, A=1, P=8, rot=64, out=f, ldo=256: lib.dspark_rope_append_q8(  # noqa: E731
        q, ldq, f, ldk, f, 128, dt, R, T, Hq, f, A, f, P, rot, None, 0, ref(c), f, None, out, ldo, f, None)
    commit = lambda c, R=1, T=2, new=g: lib.dspark_cache_commit_q8(ref(c), f, f, f, R, T, new, f, None)  # noqa: E731
    read = lambda c, n=f, R=1, S=2, dt=0, k=f, v=g, ld=128, st=f: lib.dspark_cache_read_q8(ref(c), None, n, R, S, dt, k, v, ld, st, None)  # noqa: E731
    good = _cache(ds)
    for bad in BAD_CACHES:
        c = _cache(ds, **bad)
        assert att(c) == rope(c) == commit(c) == read(c) == EINVAL, bad
    assert att(None) == rope(None) == commit(None) == read(None) == EINVAL
    for bad in (dict(n_layers=0), dict(layer_stride=-1), dict(scale_layer_stride=-1)):
        assert commit(_cache(ds, **bad)) == EINVAL
    for kw in (dict(q=None), dict(ldq=255), dict(dt=2), dict(R=-1), dict(R=1025), dict(T=0), dict(T=513), dict(Hq=3), dict(Hq=0),
               dict(Hq=1026), dict(ctx=None), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0),
               dict(cap=float("nan")), dict(out=None), dict(ldo=255), dict(st=None), dict(q=ctypes.c_void_p(257)), dict(dt=1, q=ctypes.c_void_p(258))):
        assert att(good, **kw) == EINVAL, kw
    for kw in (dict(w=None), dict(wn=100), dict(w=ctypes.c_void_p(260))):
        assert att(good, **kw) == EWORKSPACE, kw
    for kw in (dict(q=None), dict(ldq=200), dict(ldk=100), dict(dt=3), dict(T=0), dict(Hq=5), dict(A=0), dict(A=9), dict(P=0), dict(rot=0),
               dict(rot=3), dict(rot=66), dict(out=None), dict(ldo=200), dict(ldo=512, out=f), dict(R=2 ** 31, T=2)):
        assert rope(good, **kw) == EINVAL, kw
    for kw in (dict(R=65536), dict(T=0), dict(T=513), dict(new=None), dict(new=f)):
        assert commit(good, **kw) == EINVAL, kw
    for kw in (dict(n=None), dict(R=-1), dict(S=0), dict(dt=2), dict(k=None), dict(v=None), dict(v=f), dict(ld=127), dict(st=None), dict(R=2 ** 31),
               dict(dt=1, k=ctypes.c_void_p(258))):
        assert read(good, **kw) == EINVAL, kw
    ver = lambda p=f, ldp=8, q=None, ldq=0, V=8, tok=f, ua=f, ud=f, R=1, T=2, out=f, n=f, path=f, st=f: lib.dspark_tree_verify(  # noqa: E731
        p, ldp, q, ldq, V, tok, None, None, ua, ud, R, T, out, n, path, st, None)
    for kw in (dict(p=None), dict(ldp=7), dict(q=f, ldq=7), dict(V=0), dict(V=2 ** 30 + 1, ldp=2 ** 31), dict(tok=None), dict(ua=None), dict(ud=None),
               dict(R=-1), dict(R=2 ** 31), dict(T=0), dict(T=513), dict(out=None), dict(n=None), dict(path=None), dict(st=None),
               dict(p=ctypes.c_void_p(258)), dict(ua=ctypes.c_void_p(260))):
        assert ver(**kw) == EINVAL, kw


def test_empty_batches_launch_nothing(ds):
    lib, c = ds.lib(), ctypes.byref(_cache(ds))
    assert lib.dspark_rope_append_q8(None, 256, None, 128, None, 128, 0, 0, 2, 4, None, 1, None, 8, 64, None, 0, c, None, None, None, 256,
                                     None, None) == 0
    assert lib.dspark_tree_attention_q8(None, 256, 0, 0, 2, 4, c, None, None, None, 0.1, 0.0, None, 256, None, None, 0, None, None) == 0
    assert lib.dspark_cache_commit_q8(c, None, None, None, 0, 2, None, None, None) == 0
    assert lib.dspark_cache_read_q8(c, None, None, 0, 2, 0, None, None, 128, None, None) == 0
    assert lib.dspark_tree_verify(None, 8, None, 0, 8, None, None, None, None, None, 0, 2, None, None, None, None, None) == 0


def test_workspace(ds):
    for T, Hq, H, D in ((1, 8, 8, 8), (64, 32, 4, 128), (512, 64, 1, 256), (13, 12, 4, 80)):
        n = ds.dspark_workspace_size(ds.OP_TREE_ATTENTION_Q8, 3, T, Hq * D, H)
        rows = T * Hq // H
        assert n >= 2 * 148 * min(rows, 256) * (D * 4 + 16) and n >= 4 * 148 * min(rows, 64) * (D * 4 + 16)
    assert ds.dspark_workspace_size(ds.OP_TREE_ATTENTION_Q8, 0, 4, 256, 2) == 0


R, T, H, D, PAGE = 3, 2, 2, 64, 16


def _fits(ds, **kw):
    """Tensors of the host that fit together: the calls get as far as the check that they are the device's."""
    v = dict(cache=ds.q8_cache(8, PAGE, H, D, dtype=torch.int8, device="cpu"), table=torch.zeros((R, 4), dtype=torch.int32),
             q=torch.zeros((R, T, H, D)), n=torch.zeros(R, dtype=torch.int32), pos=torch.zeros((R, T), dtype=torch.int32))
    v.update(kw)
    return v


def _calls(ds, v):
    return (lambda: ds.dspark_rope_append_q8(v["q"], v["q"], v["q"], v["pos"], torch.zeros(4, D), v["cache"], v["table"], v["n"]),
            lambda: ds.dspark_tree_attention_q8(v["q"], v["cache"], v["table"], v["n"]),
            lambda: ds.dspark_cache_commit_q8(v["cache"], v["table"], v["n"], v["pos"], v["n"]),
            lambda: ds.dspark_cache_read_q8(v["cache"], v["table"], v["n"], S=3))


def test_the_binding_refuses_what_does_not_fit(ds):
    for call in _calls(ds, _fits(ds)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
    k, v, ks, vs = ds.q8_cache(8, PAGE, H, D, dtype=torch.int8, device="cpu")
    u8 = torch.uint8
    for cache, why in (((k, v[:, :, :1], ks, vs), "one shape"), ((k.float(), v.float(), ks, vs), "codes are"), ((k, v.view(torch.float8_e4m3fn), ks, vs), "one shape"),
                       ((k.transpose(-1, -2), v.transpose(-1, -2), ks, vs), "unit column stride"), ((k, v, ks[:7], vs[:7]), "scales"),
                       ((k, v, ks, vs.contiguous()), "scales"), ((k, v, ks.to(torch.int8), vs), "scales"),
                       ((k, v, *(torch.ones((8, PAGE, 2, H), dtype=u8).transpose(-1, -2) for _ in range(2))), "block stride"),
                       ((k[0], v[0], ks[0], vs[0]), "codes \\[")):
        for call in _calls(ds, _fits(ds, cache=cache)):
            with pytest.raises((ValueError, TypeError), match=why):
                call()
    for call in _calls(ds, _fits(ds, table=torch.arange(4).int()[None].expand(R, 4))):
        with pytest.raises(ValueError, match="rows overlap"):
            call()
    for call in _calls(ds, _fits(ds, table=torch.zeros((R, 4), dtype=torch.int64))):
        with pytest.raises(ValueError, match="int32 page table"):
            call()
    for bad in (dict(q=torch.zeros((R, T, H, D + 8))), dict(q=torch.zeros((R + 1, T, H, D)))):
        for call in _calls(ds, _fits(ds, **bad))[:2]:
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError, match="S, the rows"):
        ds.dspark_cache_read_q8((k, v, ks, vs), torch.zeros((R, 4), dtype=torch.int32), torch.zeros(R, dtype=torch.int32))
    with pytest.raises(TypeError):
        ds.q8_cache(2, 2, 2, 64, dtype=torch.int16, device="cpu")


def test_verify_refuses_what_does_not_fit(ds):
    p, tok, u = torch.zeros((R, T, 9)), torch.zeros((R, T), dtype=torch.int32), torch.zeros((R, T), dtype=torch.float64)
    ok = dict(p=p, tokens=tok, parent=None, u_accept=u, u_draw=u[:, 0].contiguous())
    with pytest.raises(ValueError, match="device tensors"):
        ds.dspark_tree_verify(**ok)
    monkey = ds._binding._p
    ds._binding._p = lambda t: None if t is None else 16      # past that check, to the others
    try:
        for bad in (dict(p=p.double()), dict(p=p[:2]), dict(q=p[:, :, :8]), dict(u_accept=u.float()), dict(u_accept=u[:, :1]),
                    dict(u_draw=u[:, 0].contiguous().float()), dict(tokens=tok.long()), dict(parent=tok[:2]), dict(n_nodes=tok),
                    dict(p=torch.zeros((R, 9, T)).transpose(1, 2))):
            with pytest.raises(ValueError):
                ds.dspark_tree_verify(**{**ok, **bad})
    finally:
        ds._binding._p = monkey
