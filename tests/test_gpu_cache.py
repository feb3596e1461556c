"""GPU parity of dspark_rope_append and dspark_cache_commit against the oracle. Rotated values: two
float32 products and a sum, so within 3 * 2^-24 of |x1 c| + |x2 s|, plus half a unit of bf16 (2^-8
relative) where the result is bf16; values and moved rows: equal."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

EINVAL, ERANGE = 1, 2
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def paged(gen, R, slots, page, H, D, dtype, layers=None, order="phtd"):
    """Page tables in random order over a pool with spare pages, and k, v of [layers, pages, page, H, D]
    in one of several memory orders."""
    per = -(-slots // page)
    table = torch.randperm(R * per + 2, generator=gen)[:R * per].int().reshape(R, per).cuda()
    dims = {"l": layers or 1, "p": R * per + 2, "t": page, "h": H, "d": D}
    order = ("l" + order) if "l" not in order else order
    at = [order.index(x) for x in "lpthd"]
    make = lambda: torch.randn([dims[x] for x in order], generator=gen).to(dtype).cuda().permute(at)  # noqa: E731
    k, v = make(), make()
    return table, (k if layers else k[0]), (v if layers else v[0])


def slots_of(cache, table, r, n):
    """The first n slots of request r, [..., n, H, D]."""
    page = cache.shape[-3]
    s = torch.arange(n, device="cuda")
    return cache[..., table[r].long()[s // page], s % page, :, :]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,T,Hq,H,D,rot,page,inter,axes", [
    (3, 1, 4, 2, 128, 128, 16, False, 1),
    (2, 9, 6, 2, 80, 40, 24, False, 3),          # 20 pairs: the 4-wide path
    (2, 5, 4, 4, 64, 64, 8, True, 3),
    (1, 7, 3, 1, 72, 36, 5, False, 2),           # 18 pairs: element by element
    (1, 6, 2, 1, 24, 6, 7, True, 1),
    (700, 3, 2, 1, 64, 64, 16, False, 1),        # more rows than four a block need
    (1, 301, 8, 8, 256, 256, 64, False, 4)])
def test_rope_append(dtype, R, T, Hq, H, D, rot, page, inter, axes):
    import dspark_draft_selection_gb300 as ds
    gen = torch.Generator().manual_seed(R * 100 + T + D)
    dt = TYPES[dtype]
    lens = torch.randint(0, 40, (R,), generator=gen).int()
    n = torch.randint(0, T + 1, (R,), generator=gen).int()
    n[0] = T
    order = "phtd" if T % 2 else "pthd"
    table, kc, vc = paged(gen, R, 40 + T, page, H, D, dt, order=order)
    k0, v0 = kc.clone(), vc.clone()
    qkv = torch.randn((R, T, Hq + 2 * H, D), generator=gen).to(dt).cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    P = 500
    ang = torch.arange(P).double()[:, None] * 50.0 ** (-torch.arange(rot // 2).double() / (rot // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    pos = torch.randint(0, P, (R, T, axes), generator=gen).int()
    for r in range(R):
        pos[r, n[r]:] = -77                                  # slots past the nodes hold anything
    axis = torch.randint(0, axes, (rot // 2,), generator=gen).int()
    pos_d = pos.cuda() if axes > 1 else pos[:, :, 0].contiguous().cuda()
    qo, st = ds.dspark_rope_append(q, k, v, pos_d, cs, kc, vc, table, lens.cuda(), axis=axis.cuda(), n_nodes=n.cuda(),
                                   interleaved=inter)
    assert ds.read_status(st) == 0
    table_h, csh, half = table.cpu(), f64(cs), 2.0 ** -8 if dtype == "bf16" else 0.0
    got_k, got_v = f64(kc), f64(vc)
    want_k, want_v = f64(k0), f64(v0)

    def near(got, x, c, s):
        want = tree.rope(x, c, s, inter)
        room = tree.rope(np.abs(x), np.abs(c), -np.abs(s), inter)             # |x1 c| + |x2 s| on the first columns
        other = tree.rope(np.abs(x), np.abs(c), np.abs(s), inter)
        tol = 3 * 2.0 ** -24 * np.maximum(room, other) + half * np.abs(want) * (1 + 2.0 ** -14)
        assert np.all(np.abs(got - want) <= tol), np.abs(got - want).max()

    for r in list(range(min(R, 6))) + [R - 1]:
        for i in range(T):
            if i >= n[r]:
                assert not qo[r, i].any()
                continue
            f = np.arange(rot // 2)
            p = pos[r, i].numpy()[axis.numpy()]
            c, s = csh[p, f], csh[p, rot // 2 + f]
            near(f64(qo[r, i]), f64(q[r, i]), c, s)
            at = int(lens[r]) + i
            near(got_k[table_h[r, at // page], at % page], f64(k[r, i]), c, s)
    for r in range(R):
        for i in range(int(n[r])):
            at = int(lens[r]) + i
            e = int(table_h[r, at // page]), at % page
            want_v[e] = f64(v[r, i])
            want_k[e] = got_k[e]                              # checked above
    np.testing.assert_array_equal(got_v, want_v)
    np.testing.assert_array_equal(got_k, want_k)              # nothing else was written


def _small(dt=torch.bfloat16, T=4, H=2, D=64):
    gen = torch.Generator().manual_seed(1)
    table, kc, vc = paged(gen, 1, 32, 8, H, D, dt)
    mk = lambda h: torch.randn((1, T, h, D), generator=gen).to(dt).cuda()  # noqa: E731
    pos = torch.arange(T).int()[None].cuda()
    cs = torch.cat([torch.ones(64, D // 2), torch.zeros(64, D // 2)], 1).cuda()
    return table, kc, vc, mk(2 * H), mk(H), mk(H), pos, cs, torch.tensor([3], dtype=torch.int32, device="cuda")


def test_rope_in_place_and_unaligned_rows():
    import dspark_draft_selection_gb300 as ds
    table, kc, vc, q, k, v, pos, cs, ctx = _small()
    want, _ = ds.dspark_rope_append(q, k, v, pos + 5, torch.cat([cs[:, :32] * 0.5, cs[:, :32] * 0.25], 1), kc, vc, table, ctx)
    keys = kc.clone()
    buf = torch.zeros(1 + q.numel(), dtype=q.dtype, device="cuda")   # two bytes off any 16-byte boundary
    q1 = buf[1:].view(q.shape)
    q1.copy_(q)
    got, st = ds.dspark_rope_append(q1, k, v, pos + 5, torch.cat([cs[:, :32] * 0.5, cs[:, :32] * 0.25], 1), kc, vc, table,
                                    ctx, out=q1)
    assert ds.read_status(st) == 0 and got.data_ptr() == q1.data_ptr()
    assert torch.equal(got, want) and torch.equal(kc, keys) and buf[0] == 0


def test_rope_reports_bad_pages_positions_and_counts():
    import dspark_draft_selection_gb300 as ds
    table, kc, vc, q, k, v, pos, cs, ctx = _small()
    k0 = kc.clone()
    for bad in (-1, kc.shape[0], 2 ** 31 - 1):
        t2 = torch.full_like(table, bad)
        qo, st = ds.dspark_rope_append(q, k, v, pos, cs, kc, vc, t2, ctx)
        assert ds.read_status(st) == ERANGE and torch.equal(kc, k0) and torch.equal(qo, q)
    _, st = ds.dspark_rope_append(q, k, v, pos, cs, kc, vc, table[:, :1].contiguous(), ctx + 5)   # past the table's row
    assert ds.read_status(st) == ERANGE and torch.equal(kc, k0)
    for p in (-1, 64):
        qo, st = ds.dspark_rope_append(q, k, v, torch.full_like(pos, p), cs, kc.clone(), vc.clone(), table, ctx)
        assert ds.read_status(st) == ERANGE and torch.equal(qo, q)           # position 0 turns by nothing here
    _, st = ds.dspark_rope_append(q, k, v, pos, cs, kc.clone(), vc.clone(), table, ctx,
                                  axis=torch.ones(32, dtype=torch.int32, device="cuda"))
    assert ds.read_status(st) == ERANGE
    for count in (-1, 5):
        qo, st = ds.dspark_rope_append(q, k, v, pos, cs, kc, vc, table, ctx,
                                       n_nodes=torch.tensor([count], dtype=torch.int32, device="cuda"))
        assert ds.read_status(st) == EINVAL and torch.equal(kc, k0) and not qo.any()


def test_rope_refusals():
    import dspark_draft_selection_gb300 as ds
    table, kc, vc, q, k, v, pos, cs, ctx = _small()
    call = lambda **o: ds.dspark_rope_append(**{**dict(q=q, k=k, v=v, pos=pos, cos_sin=cs, k_cache=kc, v_cache=vc,  # noqa: E731
                                                       page_table=table, ctx_len=ctx), **o})
    with pytest.raises(ds.DsparkError):                      # more rotated columns than there are
        call(cos_sin=torch.zeros((4, 66), device="cuda"))
    with pytest.raises(ds.DsparkError):
        call(pos=torch.zeros((1, 4, 9), dtype=torch.int32, device="cuda"))
    with pytest.raises(ds.DsparkError):                      # three query heads over two key heads
        call(q=q[:, :, :3])
    with pytest.raises(TypeError):
        call(q=q.float())
    with pytest.raises(ValueError):
        call(v_cache=vc.permute(0, 2, 1, 3))
    with pytest.raises(ValueError):
        call(q=q.transpose(1, 2))
    with pytest.raises(ValueError):
        call(ctx_len=ctx.long())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,T,L,H,D,page,order", [(1, 2, 1, 1, 8, 1, "phtd"), (3, 16, 2, 2, 64, 16, "pthd"),
                                                  (5, 40, 3, 3, 80, 7, "phtd"), (2, 512, 2, 1, 128, 64, "pthd"),
                                                  (2, 64, 2, 8, 128, 24, "plhtd")])
def test_commit(dtype, R, T, L, H, D, page, order):
    import dspark_draft_selection_gb300 as ds
    gen = torch.Generator().manual_seed(R + T + D)
    lens = torch.randint(0, 30, (R,), generator=gen).int()
    table, kc, vc = paged(gen, R, 30 + T, page, H, D, TYPES[dtype], layers=L, order=order)
    path = torch.full((R, T), -1, dtype=torch.int32)
    acc = torch.zeros(R, dtype=torch.int32)
    for r in range(R):
        a = int(torch.randint(0, T, (1,), generator=gen)) if r else T - 1 - T // 3
        p = torch.randperm(T - 1, generator=gen)[:a].sort().values + 1       # any rising path: moves overlap
        path[r, 0], path[r, 1:a + 1], acc[r] = 0, p.int(), a
    if R > 2:
        acc[2] = -1
    k0, v0 = kc.clone(), vc.clone()
    new, st = ds.dspark_cache_commit(kc, vc, table, lens.cuda(), path.cuda(), acc.cuda())
    assert ds.read_status(st) == 0
    for c, c0 in ((kc, k0), (vc, v0)):
        want = c0.clone()
        for r in range(R):
            rows = slots_of(c0, table, r, int(lens[r]) + T)
            for layer in range(L):
                got = tree.commit(f64(rows[layer]), int(lens[r]), path[r].tolist(), int(acc[r]))
                s = torch.arange(int(lens[r]) + T, device="cuda")
                want[layer][table[r].long()[s // page], s % page] = torch.from_numpy(got).to(c.dtype).cuda()
        assert torch.equal(c, want)
    assert new.cpu().tolist() == [int(c) + int(a) + 1 for c, a in zip(lens, acc)]


def test_commit_of_a_chain_moves_nothing_and_bad_paths_stay():
    import dspark_draft_selection_gb300 as ds
    gen = torch.Generator().manual_seed(3)
    table, kc, vc = paged(gen, 1, 32, 8, 2, 64, torch.bfloat16, layers=2)
    ctx = torch.tensor([5], dtype=torch.int32, device="cuda")
    k0 = kc.clone()
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    new, st = ds.dspark_cache_commit(kc, vc, table, ctx, None, one(6), T=8)
    assert int(new) == 12 and ds.read_status(st) == 0 and torch.equal(kc, k0)
    for path, acc in (([0, 3, 2, -1], 2), ([0, 4, -1, -1], 1), ([-1, 2, 3, -1], 2), ([0, 1, 2, 3], 4), ([0, 0, 2, 3], 3)):
        new, st = ds.dspark_cache_commit(kc, vc, table, ctx, one(path), one(acc))
        assert ds.read_status(st) == EINVAL and int(new) == 5 and torch.equal(kc, k0)
    bad = torch.full_like(table, -1)
    new, st = ds.dspark_cache_commit(kc, vc, bad, ctx, one([0, 3, -1, -1]), one(1))
    assert ds.read_status(st) == ERANGE and torch.equal(kc, k0)
    with pytest.raises(ds.DsparkError):
        ds.dspark_cache_commit(kc, vc, table, ctx, one([0] * 513), one(1))
    with pytest.raises(ds.DsparkError):                      # the new lengths may not overwrite what is read
        ds.dspark_cache_commit(kc, vc, table, ctx, one([0, 3]), one(1), out=ctx)
    with pytest.raises(ValueError):
        ds.dspark_cache_commit(kc, vc[:, :, :4], table, ctx, one([0, 3]), one(1))


def test_append_past_two_to_the_31_elements():
    """A page whose offset does not fit 32 bits: written by append, moved by commit."""
    import dspark_draft_selection_gb300 as ds
    H, D, page = 8, 128, 64
    pages = (2 ** 31 // (page * H * D)) + 40
    kc = torch.zeros((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    gen = torch.Generator().manual_seed(4)
    q = torch.randn((1, 4, H, D), generator=gen).bfloat16().cuda()
    cs = torch.cat([torch.ones(8, D // 2), torch.zeros(8, D // 2)], 1).cuda()
    table = torch.tensor([[pages - 1, pages - 20]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([62], dtype=torch.int32, device="cuda")
    pos = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    _, st = ds.dspark_rope_append(q, q, q, pos, cs, kc, vc, table, ctx)
    assert ds.read_status(st) == 0
    for c in (kc, vc):
        assert torch.equal(c[pages - 1, 62:], q[0, :2]) and torch.equal(c[pages - 20, :2], q[0, 2:])
        assert int((c[:pages - 20] != 0).sum()) == 0
    path = torch.tensor([[0, 2, 3, -1]], dtype=torch.int32, device="cuda")
    _, st = ds.dspark_cache_commit(kc, vc, table, ctx, path, torch.tensor([2], dtype=torch.int32, device="cuda"))
    assert ds.read_status(st) == 0
    assert torch.equal(kc[pages - 1, 63], q[0, 2]) and torch.equal(vc[pages - 20, 0], q[0, 3])
