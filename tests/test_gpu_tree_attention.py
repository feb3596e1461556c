"""GPU parity of dspark_tree_attention against the float64 oracle.

Tolerances. A score's float32 sum of D products is off by at most (D + 8) 2^-24 of scale sum |q||k|; a
softmax weight then by twice that (its own score and the sum's), plus 2^-20 for the exponentials and the
running rescale and len 2^-24 for the sums; the cap adds 2^-20 of itself (the tanh from exponentials). The
result is a weighted mean of v, so it is off by those times sum p |v|. bf16 on the tensor cores: each
weight is rounded once more (2^-8 of it, bf16 having eight significant bits) and the result once (2^-8)."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.gpu_util import dev
from tests.test_gpu_cache import f64, paged, slots_of
from tests.test_gpu_tree import random_trees

pytestmark = pytest.mark.gpu

EINVAL, ERANGE, ETIMEOUT = 1, 2, 6


class Case:
    def __init__(self, seed, T, Hq, H, D, page, ctx, n=None, dtype="bf16", order="pthd", mask="tree", scale=None, softcap=0.0):
        self.gen = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.T, self.Hq, self.H, self.D, self.page, self.dtype = T, Hq, H, D, page, dtype
        self.R = R = len(ctx)
        self.ctx, self.n = ctx, [T] * R if n is None else n
        self.scale, self.softcap = (D ** -0.5 if scale is None else scale), softcap
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.table, self.k, self.v = paged(self.gen, R, max(ctx) + T, page, H, D, dt, order=order)
        qkv = torch.randn((R, T, Hq + 2 * H, D), generator=self.gen).to(dt).cuda()
        self.q = qkv[:, :, :Hq]
        if mask == "tree":
            parent = random_trees(self.rng, R, T, 5)
            self.sees = np.stack([tree.tree_mask(parent[r], self.n[r])[0] for r in range(R)])
        elif mask == "any":                                  # any pattern, empty rows among it
            self.sees = self.rng.random((R, T, T)) < 0.4
            self.sees[:, ::3] = False
        elif mask == "block":
            self.sees = np.ones((R, T, T), bool)
        else:
            self.sees = np.broadcast_to(np.tri(T, dtype=bool), (R, T, T))
        self.mask = None if mask == "chain" else dev(tree.words(self.sees))

    def run(self, **kw):
        import dspark_draft_selection_gb300 as ds
        self.out, self.lse, self.status = ds.dspark_tree_attention(
            self.q, self.k, self.v, self.table, torch.tensor(self.ctx, dtype=torch.int32, device="cuda"), mask=self.mask,
            n_nodes=torch.tensor(self.n, dtype=torch.int32, device="cuda"), scale=self.scale, softcap=self.softcap, **kw)
        torch.cuda.synchronize()
        return self

    def check(self, rows=None, status=0):
        assert int(self.status) == status
        T, D = self.T, self.D
        for r in range(self.R):
            c, n = self.ctx[r], self.n[r]
            i = np.arange(T) if rows is None else np.array(rows)
            sees = np.concatenate([np.ones((T, c), bool), self.sees[r][:, :n]], 1)
            sees[n:] = False
            k, v = (f64(slots_of(x, self.table, r, c + n)) for x in (self.k, self.v))
            want, lse, mag, big = tree.attention(f64(self.q[r])[i], k, v, sees[i], self.scale, self.softcap)
            eps = 2 * (D + 8) * 2.0 ** -24 * big + 2.0 ** -20 + (c + n) * 2.0 ** -24 + 2.0 ** -20 * self.softcap
            half = 2.0 ** -8 * (1 + 2.0 ** -7) if self.dtype == "bf16" else 0.0
            got, got_lse = f64(self.out[r])[i], f64(self.lse[r])[i]
            fin = np.isfinite(want)
            tol = (eps[..., None] + half) * mag + half * np.abs(want) + 1e-30
            assert np.all(np.isfinite(got) == fin), np.argwhere(np.isfinite(got) != fin)[:5]
            bad = np.abs(got - want)[fin] > tol[fin]
            assert not bad.any(), (r, int(bad.sum()), (np.abs(got - want)[fin] / tol[fin]).max())
            np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
            ok = np.isfinite(lse)
            assert np.all(np.isneginf(got_lse) == np.isneginf(lse))
            assert np.all(np.abs(got_lse[ok] - lse[ok]) <= (eps + 2.0 ** -22 * (1 + np.abs(lse)))[ok])
        return self


SHAPES = [
    # T, Hq, H, D, page, committed lengths, node counts
    (1, 4, 4, 128, 16, [0, 1, 127, 128, 129], None),          # single tokens, one query head per key head
    (1, 8, 1, 64, 64, [300], None),                           # multi-query
    (8, 8, 2, 128, 64, [120, 121, 0, 1000], [8, 7, 8, 0]),    # the nodes end at and cross a tile's end
    (13, 6, 2, 80, 24, [37, 500], [13, 2]),                   # three query heads, 80 columns, boxes of eight
    (5, 4, 2, 40, 8, [9, 255], None),                         # fewer columns than a chunk
    (33, 8, 2, 128, 48, [130, 77], [33, 20]),                 # 132 rows: two groups of rows
    (64, 8, 2, 96, 128, [250, 3], [64, 50]),                  # 256 rows
    (100, 12, 4, 128, 32, [200], None),                       # 300 rows: two row groups, the second not full
    (200, 4, 2, 64, 16, [90], [190]),                         # nodes over several tiles
    (512, 2, 1, 64, 128, [5], None),                          # the widest tree
    (3, 5, 5, 8, 256, [700], None),                           # the smallest head
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_shapes(shape, dtype, softcap):
    T, Hq, H, D, page, ctx, n = shape
    Case(T + D, T, Hq, H, D, page, ctx, n, dtype, softcap=softcap).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,order", [(192, 16, "pthd"), (256, 32, "phtd"), (136, 7, "pthd"), (128, 5, "phtd"), (64, 1, "pthd")])
def test_heads_above_128_columns_and_odd_pages(D, page, order, dtype):
    Case(D + page, 9, 4, 2, D, page, [60, 0, 191], [9, 9, 4], dtype, order).run().check()


@pytest.mark.parametrize("mask", ["any", "block", "chain"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,ctx", [(7, [0, 3]), (70, [0, 200]), (150, [0, 60])])
def test_masks(mask, dtype, T, ctx):
    """Any pattern, with rows that see no node (and with nothing committed: nothing at all), blocks and chains."""
    Case(T, T, 4, 2, 64, 16, ctx, [T, T - 2], dtype, mask=mask, order="phtd").run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq", [(6, 4), (80, 4)])
def test_long_ragged_contexts_are_split_and_joined(dtype, T, Hq):
    """Contexts from nothing to thousands of tokens over every block of the GPU."""
    c = Case(T + 1, T, Hq, 2, 64, 64, [7000, 0, 1, 129, 2600], None, dtype, mask="chain").run()
    c.check(rows=[0, 1, T // 2, T - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [0.0, 30.0, 200.0])
@pytest.mark.parametrize("T", [1, 3, 90])                    # one tile of rows, two
def test_one_key_gives_its_value(dtype, softcap, T):
    """Nothing committed and nodes that see themselves alone: the weight is 1, so the result is v, whatever the score."""
    c = Case(T, T, 4, 2, 64, 16, [0, 0], None, dtype, mask="block", scale=2.0, softcap=softcap)
    c.sees = np.broadcast_to(np.eye(T, dtype=bool), (2, T, T))
    c.mask = dev(np.ascontiguousarray(tree.words(c.sees)))
    c.run()
    assert int(c.status) == 0
    for r in range(2):
        v = slots_of(c.v, c.table, r, T)
        assert torch.equal(c.out[r], v.repeat_interleave(2, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_maxima_that_keep_rising(dtype):
    """Keys that grow along the cache move the running maximum at every tile; the mean of v keeps its accuracy."""
    c = Case(5, 4, 4, 2, 64, 32, [1500], None, dtype, mask="chain")
    grow = torch.linspace(0.01, 12.0, 1504, device="cuda")
    s = torch.arange(1504, device="cuda")
    at = c.table[0].long()[s // 32], s % 32
    c.k[at] = (c.k[at].float() * grow[:, None, None]).to(c.k.dtype)
    c.run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [0.0, 200.0])
@pytest.mark.parametrize("T,Hq", [(4, 4), (90, 4)])        # one tile of rows, two
def test_maxima_that_leap(dtype, softcap, T, Hq):
    """Scores that jump by tens and hundreds of log2 units from one key to the next, at the places in a tile and
    in the order where the reference of the weights has to follow, and that fall as far again."""
    c = Case(6, T, Hq, 2, 64, 32, [1500], None, dtype, mask="chain", scale=0.25, softcap=softcap)
    c.q[:] = c.q.sign() * 0.5                                # every query's score of a key along its own signs is large
    s = torch.arange(1500, device="cuda")
    at = c.table[0].long()[s // 32], s % 32
    c.k[at] = (c.k[at].float() * 0.05).to(c.k.dtype)
    for j, size in ((5, 8.0), (40, -30.0), (131, 20.0), (140, 40.0), (255, 45.0), (256, 70.0), (300, 75.0), (383, 10.0),
                    (640, 130.0), (655, 190.0), (700, 60.0), (1279, 191.0), (1290, -200.0)):
        i = (j * 7) % T                                      # along another node's query each time
        for h in range(2):
            c.k[c.table[0].long()[j // 32], j % 32, h] = (c.q[0, i, h * (Hq // 2)].float() * size / 4).to(c.k.dtype)
    c.run().check(rows=None if T < 10 else [(j * 7) % T for j in (5, 131, 255, 256, 640, 655, 1279)] + [0, 1, T - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("T,ctx", [(11, 100), (70, 190), (40, 88)])
def test_what_is_not_seen_has_no_effect(dtype, junk, T, ctx):
    """Slots past the nodes, pages of nobody, and nodes that a row does not see hold junk."""
    c = Case(T, T, 8, 2, 64, 16, [ctx], [T - 3], dtype)
    used = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    s = torch.arange(ctx + T - 3, device="cuda")
    used[c.table[0].long()[s // 16], s % 16] = True
    c.k[~used], c.v[~used] = junk, junk
    c.run().check()
    for j in (2, T - 5):                                     # nodes that some rows see and others do not
        at = int(c.table[0, (ctx + j) // 16]), (ctx + j) % 16
        for buf, col in ((c.k, 5), (c.v, 7)):
            keep = buf[at].clone()
            buf[at][:, col] = junk
            c.run()
            assert int(c.status) == 0
            blind = [i for i in range(T) if not c.sees[0, i, j]]
            assert blind
            c.check(rows=blind)
            if junk != 3e38 and buf is c.v:                  # who sees it gets it
                for i in range(T - 3):
                    if c.sees[0, i, j]:
                        assert torch.all(~torch.isfinite(c.out[0, i, :, col].float()))
            buf[at] = keep


def test_rows_of_not_a_number_queries_keep_to_themselves():
    c = Case(8, 20, 4, 2, 64, 16, [150], None)
    c.q[0, 7, 2, 3] = float("nan")
    c.run()
    assert torch.isnan(c.out[0, 7, 2].float()).all() and int(c.status) == 0
    ok = [i for i in range(20) if i != 7]
    c.check(rows=ok)
    assert torch.isfinite(c.out[0, 7, [0, 1, 3]].float()).all()


def test_same_bits_every_time_on_any_stream_and_in_a_graph():
    import dspark_draft_selection_gb300 as ds
    c = Case(9, 40, 8, 2, 128, 64, [3000, 17, 900], [40, 40, 11]).run()
    first, lse = c.out.clone(), c.lse.clone()
    ctx, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.ctx, c.n))
    ws, st = ds.workspace(ds.OP_TREE_ATTENTION, 3, 40, 8 * 128, 2), ds.new_status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        c.out.fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        o, s, _ = ds.dspark_tree_attention(c.q, c.k, c.v, c.table, ctx, mask=c.mask, n_nodes=n, scale=c.scale, out=c.out, ws=ws,
                                           status=st, stream=side)
        side.synchronize()
        assert torch.equal(o, first) and torch.equal(s, lse)
    g = torch.cuda.CUDAGraph()
    out2 = torch.empty_like(first)
    with torch.cuda.graph(g):
        ds.dspark_tree_attention(c.q, c.k, c.v, c.table, ctx, mask=c.mask, n_nodes=n, scale=c.scale, out=out2, lse=False, ws=ws,
                                 status=st)
    for _ in range(3):
        out2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, first)
    ctx -= 1                                                 # lengths live on the device: the graph follows them
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out2, first) and int(st) == 0


def test_what_a_call_allocates_belongs_to_its_stream():
    """With the current stream busy, calls on another stream neither wait for it nor use memory it still works on."""
    import dspark_draft_selection_gb300 as ds
    c = Case(10, 12, 8, 2, 64, 16, [200, 33], None).run()
    want, want_lse = c.out.clone(), c.lse.clone()
    ctx, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (c.ctx, c.n))
    side = torch.cuda.Stream()
    places = torch.arange(70, device="cuda", dtype=torch.int32)

    def on_side():
        got = [ds.dspark_tree_attention(c.q, c.k, c.v, c.table, ctx, mask=c.mask, n_nodes=n, scale=c.scale, stream=side) for _ in range(4)]
        mask, pos, st = ds.dspark_tree_mask(None, R=2, T=70, stream=side)
        with torch.cuda.stream(side):
            for out, lse, status in got:
                assert torch.equal(out, want) and torch.equal(lse, want_lse) and int(status) == 0
            assert int(st) == 0 and torch.equal(pos[0], places)

    torch.cuda.synchronize()
    on_side()                                                # the stream's memory is there: no call below has to allocate
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    on_side()
    assert not torch.cuda.current_stream().query()           # the current stream was still at it
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_past_two_to_the_31_elements(dtype):
    import dspark_draft_selection_gb300 as ds
    H, D, page = 8, 128, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pages = 2 ** 31 // (page * H * D) + 40
    k, v = (torch.empty((pages, page, H, D), dtype=dt, device="cuda") for _ in range(2))
    c = Case(3, 3, 16, H, D, page, [150], None, dtype)
    far = torch.tensor([[pages - 1, pages - 30, 3]], dtype=torch.int32, device="cuda")
    for big, small in ((k, c.k), (v, c.v)):
        for e in range(3):
            big[int(far[0, e])] = small[int(c.table[0, e])]
    c.run()
    want = c.out.clone()
    c.k, c.v, c.table = k, v, far
    c.run()
    assert int(c.status) == 0 and torch.equal(c.out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_pages_lengths_and_counts_are_reported(dtype):
    import dspark_draft_selection_gb300 as ds
    c = Case(2, 4, 4, 2, 64, 16, [100, 40], None, dtype, mask="chain").run()
    good = c.out.clone()
    keep = c.table.clone()
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1):
        c.table[0, 2] = bad                                  # slots 32..47 read as zeros
        c.run()
        assert int(c.status) == ERANGE and torch.equal(c.out[1], good[1]) and torch.isfinite(c.out.float()).all()
        c.table.copy_(keep)
    c.ctx = [10 ** 9, 40]                                    # past the table's row
    c.run()
    assert int(c.status) == ERANGE and torch.equal(c.out[1], good[1])
    c.ctx = [-5, 40]
    c.run()
    assert int(c.status) == EINVAL and not c.out[0].any() and torch.equal(c.out[1], good[1])
    c.ctx, c.n = [100, 40], [5, 4]
    c.run()
    assert int(c.status) == EINVAL and not c.out[0].any() and torch.equal(c.out[1], good[1])
    assert torch.all(c.lse[0] == -float("inf"))


def test_a_wait_that_runs_out_is_reported():
    import dspark_draft_selection_gb300 as ds
    c = Case(6, 8, 8, 2, 128, 64, [2000], None)
    try:
        ds.dspark_test_set_first_wait_polls(0)
        c.run()
        assert int(c.status) == ETIMEOUT
    finally:
        ds.dspark_test_set_first_wait_polls(0xFFFFFFFF)
    c.run().check()


def test_refusals():
    import dspark_draft_selection_gb300 as ds
    c = Case(4, 4, 4, 2, 64, 16, [50], None)
    ctx = torch.tensor([50], dtype=torch.int32, device="cuda")
    call = lambda **o: ds.dspark_tree_attention(**{**dict(q=c.q, k_cache=c.k, v_cache=c.v, page_table=c.table, ctx_len=ctx,  # noqa: E731
                                                          mask=c.mask), **o})
    assert call()[0].shape == c.q.shape
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(softcap=-1.0), dict(softcap=float("inf")),
                dict(q=c.q[:, :, :3]), dict(ws=torch.empty(1000, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ds.DsparkError):
            call(**bad)
    for bad in (dict(mask=c.mask[:, :, :0]), dict(mask=c.mask.long()), dict(ctx_len=ctx.long()), dict(v_cache=c.v[:, :8]),
                dict(q=c.q.transpose(1, 2)), dict(lse=torch.empty((1, 4), device="cuda")), dict(q=c.q[..., :32]),
                dict(page_table=c.table.long()), dict(n_nodes=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(q=c.q.float())
    with pytest.raises(ds.DsparkError):                      # 513 node slots
        ds.dspark_tree_attention(torch.zeros((1, 513, 4, 64), dtype=torch.bfloat16, device="cuda"), c.k, c.v, c.table, ctx)
