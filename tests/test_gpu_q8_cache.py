"""GPU parity of the cache in 8 bits: dspark_rope_append_q8, dspark_cache_commit_q8 and dspark_cache_read_q8 against the
oracle. Codes, scale bytes, moved rows and numbers read into float32 are equal bit for bit (the format and the rounding of every
step are defined); so are numbers read into bf16, which holds them exactly. Turned queries: float32 steps as defined, equal in float32, and in
bf16 after one rounding."""
import numpy as np
import pytest
import torch

from oracle import q8
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

EINVAL, ERANGE, ENONFINITE = 1, 2, 5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
N = 200                                                      # spare bytes before and after every buffer, which nobody may touch


def raw(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype is not torch.uint8 else t.cpu().numpy()


def paged(gen, R, slots, page, H, D, code, layers=None, order="phtd", sorder="phtd", low=121, high=132, offset=0):
    """(table, (k, v, k_scale, v_scale)): page tables in random order over a pool with spare pages, filled with random codes and
    scale bytes from [low, high], in one of several memory orders; `offset` bytes shift the codes off their alignment."""
    per = max(1, -(-slots // page))
    table = torch.randperm(R * per + 2, generator=gen)[:R * per].int().reshape(R, per).cuda()

    def make(cols, order, draw, off):
        dims = {"l": layers or 1, "p": R * per + 2, "t": page, "h": H, "d": cols}
        order = ("l" + order) if "l" not in order else order
        shape = [dims[x] for x in order]
        buf = torch.full((off + int(np.prod(shape)),), 0, dtype=torch.uint8)
        buf[off:] = draw(int(np.prod(shape)))
        t = buf.cuda()[off:].view(shape).permute([order.index(x) for x in "lpthd"])
        return t if layers else t[0]

    def codes(n):                                            # (0x7F and 0xFF are no numbers in e4m3)
        c = torch.randint(0, 256, (n,), generator=gen).to(torch.uint8)
        return torch.where((c & 127) == 127, c - 1, c) if code == "e4m3" else c

    bytes_ = lambda n: torch.randint(low, high + 1, (n,), generator=gen).to(torch.uint8)  # noqa: E731
    k, v = (make(D, order, codes, offset).view(CODES[code]) for _ in range(2))
    ks, vs = (make((D + 31) // 32, sorder, bytes_, 0) for _ in range(2))
    return table, (k, v, ks, vs)


def numbers(cache, code):
    """Keys and values of a whole cache in float64, on the GPU."""
    k, v, ks, vs = cache
    return tuple(torch.from_numpy(q8.numbers(raw(c), raw(s), code == "e4m3")).cuda() for c, s in ((k, ks), (v, vs)))


def where(table, r, slots, page):
    t = table.cpu().numpy()
    return t[r, slots // page], slots % page


APPENDS = [
    # R, T, Hq, H, D, rot, page, interleaved, axes, order, sorder, offset
    (3, 1, 4, 2, 128, 128, 16, False, 1, "phtd", "phtd", 0),
    (2, 9, 6, 2, 80, 32, 24, False, 3, "pthd", "phtd", 0),       # 80 columns: a short last block; 16 pairs: vectors
    (2, 5, 4, 4, 64, 64, 8, True, 3, "phtd", "pthd", 0),
    (1, 7, 3, 1, 72, 36, 5, False, 2, "pthd", "pthd", 0),        # 18 pairs: column by column
    (1, 6, 2, 1, 24, 6, 7, True, 1, "pthd", "phtd", 0),
    (2, 3, 2, 2, 8, 8, 4, False, 1, "phtd", "phtd", 0),
    (2, 4, 2, 1, 64, 64, 16, False, 1, "phtd", "phtd", 3),       # codes off any alignment
    (1, 3, 8, 8, 256, 200, 16, False, 4, "pthd", "phtd", 0),
    (700, 3, 2, 1, 64, 64, 16, False, 1, "phtd", "phtd", 0),     # two rows a block
]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", APPENDS)
@pytest.mark.parametrize("inplace", [False, True])
def test_append(shape, dtype, code, inplace):
    import dspark_draft_selection_gb300 as ds
    R, T, Hq, H, D, rot, page, inter, axes, order, sorder, offset = shape
    if inplace and (R > 3 or D not in (64, 72, 24)):
        pytest.skip("in place: one shape for every path")
    gen = torch.Generator().manual_seed(R * 100 + T + D)
    dt = TYPES[dtype]
    lens = torch.randint(0, 40, (R,), generator=gen).int()
    n = torch.randint(0, T + 1, (R,), generator=gen).int()
    n[0] = T
    table, cache = paged(gen, R, 40 + T, page, H, D, code, order=order, sorder=sorder, offset=offset)
    before = [c.clone() for c in cache]
    x = torch.randn((R, T, Hq + 2 * H, D), generator=gen) * 10.0 ** (4 * torch.rand((R, T, Hq + 2 * H, 1), generator=gen) - 2)
    x[0, 0, Hq:] = 0.0                                       # a row of zeros
    qkv = x.to(dt).cuda()
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    P = 500
    ang = torch.arange(P).double()[:, None] * 50.0 ** (-torch.arange(rot // 2).double() / (rot // 2))
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    pos = torch.randint(0, P, (R, T, axes), generator=gen).int()
    for r in range(R):
        pos[r, n[r]:] = -77                                  # slots past the nodes hold anything
    axis = torch.randint(0, axes, (rot // 2,), generator=gen).int()
    pos_d = pos.cuda() if axes > 1 else pos[:, :, 0].contiguous().cuda()
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    qh, kh, vh, csh, h = f(q), f(k), f(v), cs.cpu().numpy(), rot // 2
    qo, st = ds.dspark_rope_append_q8(q, k, v, pos_d, cs, cache, table, lens.cuda(), axis=axis.cuda(), n_nodes=n.cuda(), interleaved=inter,
                                      out=q if inplace else None)
    assert ds.read_status(st) == 0
    want = [raw(b).copy() for b in before]
    rows = range(R) if R < 10 else [0, 1, R // 2, R - 1]
    e4m3 = code == "e4m3"
    for r in rows:
        for i in range(T):
            if i >= n[r]:
                assert not qo[r, i].any()
                continue
            at = pos[r, i][axis.long()].numpy()
            c, s = csh[at, np.arange(h)], csh[at, h + np.arange(h)]
            wq = torch.from_numpy(q8.turn(qh[r, i], c, s, inter)).to(dt)
            assert torch.equal(qo[r, i].cpu(), wq)
            p, o = where(table, r, np.array([int(lens[r]) + i]), page)
            for b, y in ((0, q8.turn(kh[r, i], c, s, inter)), (1, vh[r, i])):
                codes, scale = q8.quantise(y, e4m3)
                want[b][p[0], o[0]], want[2 + b][p[0], o[0]] = codes, scale
    if R < 10:                                               # every other byte is what it was
        for got, w in zip(cache, want):
            np.testing.assert_array_equal(raw(got), w)
    else:
        for r in rows:
            p, o = where(table, r, np.arange(int(lens[r]), int(lens[r] + n[r])), page)
            for got, w in zip(cache, want):
                np.testing.assert_array_equal(raw(got)[p, o], w[p, o])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 72])                      # vectors; column by column (18 pairs)
def test_numbers_of_every_size_and_what_is_not_finite(code, D):
    """Blocks from the least subnormal to the largest float32, borders of the scale's rule, infinities and NaN."""
    import dspark_draft_selection_gb300 as ds
    R, T, H = 1, 24, 1
    table, cache = paged(torch.Generator().manual_seed(0), R, 40, 16, H, D, code)
    top = 448.0 if code == "e4m3" else 127.0
    y = np.random.default_rng(1).standard_normal((R, T, H, D)).astype(np.float32)
    y[0, :, 0] *= 2.0 ** np.linspace(-149, 126, T)[:, None]
    y[0, 3, 0, :32] = 0.0
    y[0, 4, 0, 0], y[0, 5, 0, 0] = top * 4, np.nextafter(np.float32(top * 4), np.float32(1e9))
    y[0, 4, 0, 1:], y[0, 5, 0, 1:] = 1.0, 1.0
    y[0, 6, 0, :3] = [3.4e38, -3.4e38, 1e-45]
    clean = y.copy()
    y[0, 7, 0, :4] = [np.nan, np.inf, -np.inf, 1.0]
    cs = torch.cat([torch.ones(1, 36), torch.zeros(1, 36)], 1)[:, 36 - D // 2:36 + D // 2].contiguous().cuda()   # turns by nothing
    zero = torch.zeros((R, T), dtype=torch.int32, device="cuda")
    for data, status in ((clean, 0), (y, ENONFINITE)):
        t = dev(data)
        _, st = ds.dspark_rope_append_q8(t.clone(), t * 0, t, zero, cs, cache, table, zero[:, 0].contiguous())
        if status == 0:                                      # (0 times NaN among the keys would report it too)
            assert ds.read_status(st) == 0
        else:
            assert ds.read_status(st) == ENONFINITE
        p, o = where(table, 0, np.arange(T), 16)
        codes, scale = q8.quantise(data[0], code == "e4m3")
        np.testing.assert_array_equal(raw(cache[1])[p, o], codes)
        np.testing.assert_array_equal(raw(cache[3])[p, o], scale)
        k, v, st = ds.dspark_cache_read_q8(cache, table, torch.tensor([T], dtype=torch.int32, device="cuda"), S=T, dtype=torch.float32)
        np.testing.assert_array_equal(v[0].cpu().numpy(), q8.numbers(codes, scale, code == "e4m3").astype(np.float32))
        assert ds.read_status(st) == 0 and torch.isfinite(v).all()


def test_append_reports_what_is_out_of_range():
    import dspark_draft_selection_gb300 as ds
    gen = torch.Generator().manual_seed(3)
    R, T, H, D, page = 4, 5, 2, 64, 8
    table, cache = paged(gen, R, 16, page, H, D, "int8")
    x = torch.randn((R, T, H, D), generator=gen).cuda()
    cs = torch.randn((9, D), generator=gen).cuda()
    pos = torch.randint(0, 9, (R, T), generator=gen).int().cuda()
    ctx = torch.tensor([3, 4, 0, 2], dtype=torch.int32, device="cuda")

    def go(table=table, ctx=ctx, pos=pos, n=None):
        c = [t.clone() for t in cache]
        q, st = ds.dspark_rope_append_q8(x, x, x, pos, cs, c, table, ctx, n_nodes=n)
        return c, q, ds.read_status(st)

    good, q, st = go()
    assert st == 0
    bad = table.clone()
    bad[1, 0], bad[2, 0] = -1, 10 ** 6                       # pages that do not exist: their rows are left out
    c, q1, st = go(bad)
    assert st == ERANGE and torch.equal(q1, q)
    for r, kept in ((0, True), (1, False), (3, True)):
        p, o = where(table, r, np.arange(int(ctx[r]), int(ctx[r]) + 4), page)
        for a, b, old in zip(c, good, cache):
            np.testing.assert_array_equal(raw(a)[p, o], (raw(b) if kept else raw(old))[p, o])
    c, _, st = go(ctx=torch.tensor([3, 13, 0, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))      # past the table's row
    assert st == ERANGE
    assert go(ctx=torch.tensor([3, -1, 0, 2], dtype=torch.int32, device="cuda"))[2] == EINVAL
    assert go(n=torch.tensor([1, 2, 6, 0], dtype=torch.int32, device="cuda"))[2] == EINVAL
    assert go(pos=pos + 9)[2] == ERANGE


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("H,D,page,layers,order,sorder,offset", [
    (2, 128, 16, 3, "phtd", "phtd", 0), (3, 80, 24, 2, "pthd", "phtd", 0), (1, 24, 5, None, "pthd", "pthd", 0),
    (2, 128, 8, 2, "lphtd", "lpthd", 0), (2, 64, 16, 2, "phtd", "phtd", 5), (9, 256, 16, 1, "pthd", "pthd", 8)])
def test_commit(code, H, D, page, layers, order, sorder, offset):
    import dspark_draft_selection_gb300 as ds
    rng = np.random.default_rng(D)
    R, T = 6, 40
    lens = rng.integers(0, 30, R).astype(np.int32)
    table, cache = paged(torch.Generator().manual_seed(D), R, 30 + T, page, H, D, code, layers, order, sorder, offset=offset)
    acc = np.array([0, -1, 5, 39, 12, 1], np.int32)
    path = np.full((R, T), -1, np.int32)
    for r, a in enumerate(acc):
        if a >= 0:
            path[r, :a + 1] = np.sort(rng.choice(T, a + 1, replace=False))
    path[5, :2] = [0, 1]                                     # nothing moves
    want = [raw(c).copy() for c in cache]
    for w, c in zip(want, cache):
        old = raw(c)
        for r, a in enumerate(acc):
            for k in range(a + 1):
                (sp, so), (dp, do) = (where(table, r, np.array([int(lens[r]) + x]), page) for x in (path[r, k], k))
                if layers:
                    w[:, dp[0], do[0]] = old[:, sp[0], so[0]]
                else:
                    w[dp[0], do[0]] = old[sp[0], so[0]]
    new, st = ds.dspark_cache_commit_q8(cache, table, dev(lens), dev(path), dev(acc))
    assert ds.read_status(st) == 0
    np.testing.assert_array_equal(new.cpu().numpy(), lens + np.maximum(acc, -1) + 1)
    for got, w in zip(cache, want):
        np.testing.assert_array_equal(raw(got), w)


def test_commit_refuses_bad_paths_and_follows_chains():
    import dspark_draft_selection_gb300 as ds
    table, cache = paged(torch.Generator().manual_seed(7), 3, 40, 8, 2, 64, "int8")
    before = [raw(c).copy() for c in cache]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx = i32([3, 4, 5])
    for path, acc in (([[0, 3, 2, -1]] * 3, [2, 0, 0]), ([[0, 1, 2, 4]] * 3, [3, 0, 0]), ([[0, 1, 2, 3]] * 3, [4, 0, 0]),
                      ([[0, 1, 2, 3]] * 3, [2 ** 31 - 1, 0, 0])):
        new, st = ds.dspark_cache_commit_q8(cache, table, ctx, i32(path), i32(acc))
        assert ds.read_status(st) == EINVAL and new.tolist()[0] == 3
        for got, w in zip(cache, before):
            np.testing.assert_array_equal(raw(got), w)
    new, st = ds.dspark_cache_commit_q8(cache, table, ctx, None, i32([3, -1, 0]), T=4)
    assert ds.read_status(st) == 0 and new.tolist() == [7, 4, 6]
    new, st = ds.dspark_cache_commit_q8(cache, table, i32([36, 40, 0]), i32([[1, 2, 3, 9]] * 3), i32([3, 1, -1]))     # 9 is no node of four
    assert ds.read_status(st) == EINVAL and new.tolist() == [36, 42, 0]
    new, st = ds.dspark_cache_commit_q8(cache, table, i32([38, 0, 0]), i32([[1, 2, 3, -1]] * 3), i32([2, -1, -1]))   # past the table
    assert ds.read_status(st) == ERANGE and new.tolist() == [41, 0, 0]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,D,page,order,sorder,offset,pad", [
    (2, 128, 16, "phtd", "phtd", 0, 0), (3, 80, 24, "pthd", "pthd", 0, 16), (1, 24, 5, "pthd", "phtd", 0, 0), (2, 64, 16, "phtd", "phtd", 1, 0),
    (2, 8, 4, "phtd", "phtd", 0, 3), (1, 256, 64, "pthd", "phtd", 0, 0)])
def test_read(code, dtype, H, D, page, order, sorder, offset, pad):
    import dspark_draft_selection_gb300 as ds
    R, S = 5, 37
    gen = torch.Generator().manual_seed(D + page)
    table, cache = paged(gen, R, 80, page, H, D, code, order=order, sorder=sorder, offset=offset, low=0, high=255)
    dt = TYPES[dtype]
    start, n = np.array([0, 7, 40, 3, 79], np.int32), np.array([37, 0, 33, 1, 1], np.int32)
    wide = [torch.full((R, S, H * D + pad), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    out = tuple(w[:, :, :H * D].unflatten(-1, (H, D)) for w in wide)
    k, v, st = ds.dspark_cache_read_q8(cache, table, dev(n), start=dev(start), out=out)
    assert ds.read_status(st) == 0
    for got, codes, scale in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        c, s = raw(codes), raw(scale)
        for r in range(R):
            p, o = where(table, r, np.arange(start[r], start[r] + n[r]), page)
            want = torch.from_numpy(q8.numbers(c[p, o], s[p, o], code == "e4m3"))
            big = want.abs() >= 2.0 ** -126                  # (below, a number may be read as 0)
            g = got[r, :n[r]].double().cpu()
            assert torch.equal(g[big], want[big]) and ((g - want).abs()[~big] <= want.abs()[~big]).all()
            assert (got[r, n[r]:] == 7.0).all()
    for w in wide:
        assert (w[:, :, H * D:] == 7.0).all()
    k2, v2, st = ds.dspark_cache_read_q8(cache, table, dev(n), start=dev(start), S=S, dtype=dt)
    assert ds.read_status(st) == 0 and torch.equal(k2[0], k[0]) and not k2[1].any()


def test_read_reports_what_is_out_of_range():
    import dspark_draft_selection_gb300 as ds
    table, cache = paged(torch.Generator().manual_seed(9), 4, 32, 8, 2, 64, "e4m3")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good, _, st = ds.dspark_cache_read_q8(cache, table, i32([32, 3, 0, 9]), S=32)
    assert ds.read_status(st) == 0
    bad = table.clone()
    bad[3, 1], bad[1, 0] = -5, 10 ** 6
    k, v, st = ds.dspark_cache_read_q8(cache, bad, i32([32, 3, 0, 9]), S=32)
    assert ds.read_status(st) == ERANGE and torch.equal(k[0], good[0]) and not k[1].any() and not k[3, 8:].any()
    assert torch.equal(k[3, :8], good[3, :8])
    k, v, st = ds.dspark_cache_read_q8(cache, table, i32([3, 3, 0, 9]), start=i32([30, 2 ** 31 - 1, 0, 0]), S=32)
    assert ds.read_status(st) == ERANGE and not k[0, 2:].any() and not k[1].any()
    for n, start in (([33, 0, 0, 1], [0, 0, 0, 0]), ([-1, 0, 0, 1], [0, 0, 0, 0]), ([3, 0, 0, 1], [-1, 0, 0, 0])):
        k, v, st = ds.dspark_cache_read_q8(cache, table, i32(n), start=i32(start), S=32)
        assert ds.read_status(st) == EINVAL and not k[0].any() and torch.equal(k[3, :1], good[3, :1])
