"""GPU parity of dspark_tree_attention_q8 against the float64 oracle, over the numbers that the codes stand for: the tolerances of
tests/test_gpu_tree_attention.py, whose cases these are (the codes' numbers are exact in bf16 and float32, so nothing is added)."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.gpu_util import dev
from tests.test_gpu_q8_cache import numbers, paged
from tests.test_gpu_tree_attention import SHAPES, Case

pytestmark = pytest.mark.gpu

EINVAL, ERANGE = 1, 2


class Q8Case(Case):
    def __init__(self, seed, T, Hq, H, D, page, ctx, n=None, dtype="bf16", code="e4m3", order="pthd", sorder="phtd", offset=0, low=114, high=121, **kw):
        super().__init__(seed, T, Hq, H, D, page, ctx, n, dtype, **kw)
        self.code = code
        self.table, self.cache = paged(self.gen, self.R, max(ctx) + T, page, H, D, code, order=order, sorder=sorder, offset=offset,
                                       low=low, high=high)
        self.k, self.v = numbers(self.cache, code)

    def run(self, **kw):
        import dspark_draft_selection_gb300 as ds
        self.out, self.lse, self.status = ds.dspark_tree_attention_q8(
            self.q, self.cache, self.table, torch.tensor(self.ctx, dtype=torch.int32, device="cuda"), mask=self.mask,
            n_nodes=torch.tensor(self.n, dtype=torch.int32, device="cuda"), scale=self.scale, softcap=self.softcap, **kw)
        torch.cuda.synchronize()
        return self


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_shapes(shape, dtype, code, softcap):
    T, Hq, H, D, page, ctx, n = shape
    Q8Case(T + D, T, Hq, H, D, page, ctx, n, dtype, code, softcap=softcap).run().check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 12, 16, 17, 24, 32])
@pytest.mark.parametrize("ctx", [[1, 63, 64, 65], [511, 0, 700, 16]])
def test_single_tokens(G, ctx, code):
    """One new token a request, from one query head per key head to more than a tensor-core tile's rows."""
    Q8Case(G, 1, 2 * G, 2, 128, 16, ctx, None, "bf16", code, mask="chain").run().check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("T,G", [(1, 4), (9, 3), (40, 2)])
def test_columns(D, T, G, code):
    Q8Case(D, T, 2 * G, 2, D, 16, [200, 31], None, "bf16", code).run().check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,page,order,offset", [(192, 16, "pthd", 0), (256, 32, "phtd", 0), (136, 7, "pthd", 0), (128, 5, "phtd", 0),
                                                 (64, 1, "pthd", 0), (64, 16, "phtd", 3), (72, 16, "phtd", 0), (128, 16, "phtd", 8)])
def test_heads_above_128_columns_odd_pages_and_odd_rows(D, page, order, offset, dtype, code):
    Q8Case(D + page, 9, 4, 2, D, page, [60, 0, 191], [9, 9, 4], dtype, code, order, offset=offset).run().check()


@pytest.mark.parametrize("sorder", ["pthd", "phtd", "tphd"])
@pytest.mark.parametrize("T", [2, 40])
def test_orders_of_the_scales(sorder, T):
    Q8Case(T, T, 8, 2, 128, 16, [300, 17], None, "bf16", "e4m3", "phtd", sorder).run().check()


@pytest.mark.parametrize("mask", ["any", "block", "chain"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,ctx", [(3, [0, 126]), (7, [0, 3]), (70, [0, 200]), (150, [0, 60])])
def test_masks(mask, dtype, T, ctx):
    """Any pattern, with rows that see no node (and with nothing committed: nothing at all), blocks and chains."""
    Q8Case(T, T, 4, 2, 64, 16, ctx, [T, T - 2], dtype, "int8", mask=mask, order="phtd").run().check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq", [(1, 8), (6, 4), (12, 8), (80, 4)])
def test_long_ragged_contexts_are_split_and_joined(dtype, T, Hq, code):
    c = Q8Case(T + 1, T, Hq, 2, 64, 64, [7000, 0, 1, 129, 2600], None, dtype, code, mask="chain").run()
    c.check(rows=sorted({0, min(1, T - 1), T // 2, T - 1}))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [0.0, 30.0, 200.0])
@pytest.mark.parametrize("T", [1, 3, 20, 90])
def test_one_key_gives_its_value(dtype, softcap, T, code):
    """Nothing committed and nodes that see themselves alone: the weight is 1, so the result is v, whatever the score."""
    c = Q8Case(T, T, 4, 2, 64, 16, [0, 0], None, dtype, code, mask="block", scale=2.0, softcap=softcap)
    c.sees = np.broadcast_to(np.eye(T, dtype=bool), (2, T, T))
    c.mask = dev(np.ascontiguousarray(tree.words(c.sees)))
    c.run().check()
    page, s = 16, torch.arange(T, device="cuda")
    for r in range(2):
        v = c.v[c.table[r].long()[s // page], s % page]
        assert torch.equal(c.out[r].double(), v.repeat_interleave(2, 1))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("T,softcap", [(1, 0.0), (5, 0.0), (5, 30.0), (40, 0.0)])
def test_maxima_that_keep_rising(T, softcap, code):
    """Scales that grow along the cache move the running maximum again and again; the mean of v keeps its accuracy."""
    c = Q8Case(5, T, 4, 2, 64, 32, [1500], None, "bf16", code, mask="chain", softcap=softcap)
    s = torch.arange(1500 + T, device="cuda")
    c.cache[2][c.table[0].long()[s // 32], s % 32] = (105 + s // 100).to(torch.uint8)[:, None, None]
    c.k, c.v = numbers(c.cache, code)
    c.run().check()


@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("softcap", [0.0, 1e-3, 1.0, 1e4])
def test_caps(T, softcap):
    Q8Case(T, T, 4, 2, 128, 16, [300, 5], None, "bf16", "int8", softcap=softcap, scale=0.3).run().check()


@pytest.mark.parametrize("T", [1, 8, 50])
def test_far_scales(T):
    """The least and the largest scale bytes among the values: numbers near both ends of float32's range."""
    for low, high in ((1, 3), (0, 0), (224, 226)):
        c = Q8Case(T, T, 4, 2, 64, 16, [70], None, "bf16", "e4m3", mask="chain")
        v = c.cache[3]
        v.copy_(torch.randint(low, high + 1, v.shape, device="cuda").to(torch.uint8))
        c.k, c.v = numbers(c.cache, "e4m3")
        c.run()
        want = [tree.attention(c.q[r].double().cpu().numpy(), *(x[c.table[r].long()[torch.arange(70 + T, device="cuda") // 16],
                                                              torch.arange(70 + T, device="cuda") % 16].cpu().numpy() for x in (c.k, c.v)),
                               np.concatenate([np.ones((T, 70), bool), np.tri(T, dtype=bool)], 1), c.scale)[0] for r in range(1)][0]
        got = c.out[0].double().cpu().numpy()
        assert np.isfinite(got).all()
        if high > 3:
            assert np.abs(got - want).max() <= 2.0 ** -6 * np.abs(want).max()
        else:                                                # subnormal numbers may be 0
            assert np.abs(got - want).max() <= 2.0 ** -6 * np.abs(want).max() + 2.0 ** -126


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("T", [3, 20, 70])
def test_scales_on_both_sides_of_2_to_the_7(T, code, head_dim):
    """Blocks of a value row, and rows of a tile, whose powers of two lie below and above what one bf16 factor reaches over E4M3 codes."""
    c = Q8Case(T, T, 4, 2, head_dim, 16, [150], None, "bf16", code, mask="chain")
    v = c.cache[3]
    v.copy_(torch.randint(128, 142, v.shape, device="cuda").to(torch.uint8))
    c.k, c.v = numbers(c.cache, code)
    c.run()
    at = torch.arange(150 + T, device="cuda")
    k, x = (t[c.table[0].long()[at // 16], at % 16].cpu().numpy() for t in (c.k, c.v))
    want, _, mag, _ = tree.attention(c.q[0].double().cpu().numpy(), k, x, np.concatenate([np.ones((T, 150), bool), np.tri(T, dtype=bool)], 1), c.scale)
    # a weight, its sum's share and the result are off by half a step of bf16 each, the weight twice that where the sum is the unrounded one
    assert (np.abs(c.out[0].double().cpu().numpy() - want) <= 2.0 ** -7 * mag + 2.0 ** -8 * np.abs(want)).all()


@pytest.mark.parametrize("T", [1, 8, 40])
def test_what_nobody_sees_changes_no_bit(T):
    """Stale codes and scales of any value behind the sequences, in unseen pages, and infinite queries of other rows."""
    c = Q8Case(T, T, 4, 2, 128, 16, [50, 3], [T, max(0, T - 1)], "bf16", "e4m3", mask="chain").run()
    first, lse = c.out.clone(), c.lse.clone()
    end = [a + b for a, b in zip(c.ctx, c.n)]
    seen = torch.zeros(c.cache[0].shape[:2], dtype=torch.bool, device="cuda")
    for r in range(2):
        s = torch.arange(end[r], device="cuda")
        seen[c.table[r].long()[s // 16], s % 16] = True
    for t, fill in zip(c.cache, (0x7F, 0xFF, 255, 255)):
        u = t.view(torch.uint8)
        u[~seen] = fill
    q = c.q.clone()
    q[1, c.n[1]:] = float("nan")
    c.q = q
    c.run()
    assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("T,Hq", [(2, 4), (4, 8), (8, 8), (40, 4)])
def test_the_largest_values_in_a_node_that_others_do_not_see(T, Hq, code):
    """The last node of a chain has values near float32's largest, all others small ones: the rows before it keep their accuracy."""
    c = Q8Case(T, T, Hq, 2, 128, 16, [70], None, "bf16", code, mask="chain")
    v = c.cache[3]
    v.copy_(torch.randint(88, 110, v.shape, device="cuda").to(torch.uint8))
    last = 70 + T - 1
    v[c.table[0, last // 16].long(), last % 16] = 245
    c.k, c.v = numbers(c.cache, code)
    c.run()
    at = torch.arange(70 + T, device="cuda")
    k, x = (t[c.table[0].long()[at // 16], at % 16].cpu().numpy() for t in (c.k, c.v))
    want, _, mag, _ = tree.attention(c.q[0].double().cpu().numpy(), k, x, np.concatenate([np.ones((T, 70), bool), np.tri(T, dtype=bool)], 1), c.scale)
    # a weight, its sum's share and the result are off by half a step of bf16 each, the weight twice that where the sum is the unrounded one
    assert (np.abs(c.out[0].double().cpu().numpy() - want) <= 2.0 ** -7 * mag + 2.0 ** -8 * np.abs(want)).all()


@pytest.mark.parametrize("T", [1, 3, 40])
def test_a_query_that_is_not_finite_stays_in_its_row(T):
    c = Q8Case(T, T, 8, 2, 64, 16, [130], None, "bf16", "int8", mask="chain").run()
    first = c.out.clone()
    q = c.q.clone()
    q[0, 0, 3, 5] = float("inf")
    c.q = q
    c.run()
    keep = torch.ones_like(first, dtype=torch.bool)
    keep[0, 0, 3] = False
    assert torch.equal(c.out[keep], first[keep])
    assert not torch.isfinite(c.out[0, 0, 3]).all()


@pytest.mark.parametrize("T", [1, 4, 40])
def test_pages_and_lengths_out_of_range(T):
    import dspark_draft_selection_gb300 as ds
    c = Q8Case(T, T, 4, 2, 64, 16, [64, 64, 64], None, "bf16", "e4m3", mask="chain").run()
    good = c.out.clone()
    table = c.table.clone()
    table[1, 2] = -1
    c.table = table
    c.run()
    assert int(c.status) == ERANGE
    assert torch.equal(c.out[0], good[0]) and torch.equal(c.out[2], good[2]) and torch.isfinite(c.out).all()
    c.table[1, 2] = 0
    cap = c.table.shape[1] * 16
    for ctx, n, code in (([64, -1, 64], [T, T, T], EINVAL), ([64, 64, 64], [T, T + 1, T], EINVAL), ([64, 64, 64], [T, -1, T], EINVAL),
                         ([64, cap, 64], [T, T, T], ERANGE), ([64, 2 ** 31 - 1, 64], [T, T, T], ERANGE)):
        out, lse, st = ds.dspark_tree_attention_q8(c.q, c.cache, c.table, torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                                                   n_nodes=torch.tensor(n, dtype=torch.int32, device="cuda"), scale=c.scale)
        # the other requests' results (the work is split otherwise, so not to the bit), and zeros for this one
        c.out, c.lse, c.status = out, lse, st
        c.ctx, c.n = [64, 0, 64], [T, 0, T]
        c.check(status=code)
        c.ctx, c.n = [64] * 3, [T] * 3


@pytest.mark.parametrize("T", [1, 7, 40])
def test_runs_give_the_same_bits_also_captured_and_on_other_streams(T):
    import dspark_draft_selection_gb300 as ds
    c = Q8Case(T, T, 8, 2, 128, 64, [5000, 40, 900], None, "bf16", "int8", mask="chain").run()
    first = c.out.clone()
    ctx = torch.tensor(c.ctx, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    out, _, st = ds.dspark_tree_attention_q8(c.q, c.cache, c.table, ctx, scale=c.scale, stream=side)
    side.synchronize()
    assert torch.equal(out, first) and ds.read_status(st) == 0
    ws = ds.workspace(ds.OP_TREE_ATTENTION_Q8, c.R, T, 8 * 128, 2)
    out, lse, st = torch.empty_like(first), torch.empty_like(c.lse), ds.new_status()
    call = lambda: ds.dspark_tree_attention_q8(c.q, c.cache, c.table, ctx, scale=c.scale, out=out, lse=lse, ws=ws, status=st)  # noqa: E731
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for k in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and ds.read_status(st) == 0
    ctx.copy_(torch.tensor([17, 0, 901], dtype=torch.int32))     # a graph follows the lengths
    g.replay()
    eager, _, _ = ds.dspark_tree_attention_q8(c.q, c.cache, c.table, ctx, scale=c.scale)
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


def test_many_requests_and_strided_queries():
    """More requests than a warp takes at once, and heads that lie among others."""
    R = 300
    rng = np.random.default_rng(1)
    ctx = rng.integers(0, 90, R).tolist()
    c = Q8Case(R, 2, 4, 2, 64, 16, ctx, None, "bf16", "e4m3", mask="chain").run()
    c.check()


@pytest.mark.parametrize("T", [1, 8, 40])
def test_pages_past_two_to_the_31_bytes(T):
    """Codes and scales whose offsets pass 32 bits."""
    H, D, page = 8, 128, 64
    pages = 2 ** 31 // (page * H * D) + 40
    codes = [torch.empty((pages, page, H, D), dtype=torch.uint8, device="cuda").view(torch.int8) for _ in range(2)]
    wide = [torch.empty((pages, H, 16, page, 4), dtype=torch.uint8, device="cuda")[:, :, 3].transpose(1, 2) for _ in range(2)]
    c = Q8Case(T, T, 16, H, D, page, [150], None, "bf16", "int8", mask="chain")
    far = torch.tensor([[pages - 1, pages - 30, 3]], dtype=torch.int32, device="cuda")
    big = (*codes, *wide)
    for b, small in zip(big, c.cache):
        for e in range(far.shape[1]):
            b[int(far[0, e])] = small[int(c.table[0, e])]
    c.run()
    want = c.out.clone()
    c.cache, c.table = big, far
    c.run()
    assert int(c.status) == 0 and torch.equal(c.out, want)


@pytest.mark.parametrize("T", [1, 6, 40, 90])
def test_a_wait_that_runs_out_is_reported(T):
    import dspark_draft_selection_gb300 as ds
    c = Q8Case(T, T, 8, 2, 128, 64, [2000], None)
    try:
        ds.dspark_test_set_first_wait_polls(0)
        c.run()
        assert int(c.status) == 6
    finally:
        ds.dspark_test_set_first_wait_polls(0xFFFFFFFF)
    c.run().check(rows=[0, T - 1])


def test_refusals():
    import dspark_draft_selection_gb300 as ds
    c = Q8Case(4, 4, 4, 2, 64, 16, [50], None)
    ctx = torch.tensor([50], dtype=torch.int32, device="cuda")
    call = lambda **o: ds.dspark_tree_attention_q8(**{**dict(q=c.q, cache=c.cache, page_table=c.table, ctx_len=ctx, mask=c.mask), **o})  # noqa: E731
    assert call()[0].shape == c.q.shape
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(softcap=-1.0), dict(softcap=float("inf")), dict(q=c.q[:, :, :3]),
                dict(ws=torch.empty(1000, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ds.DsparkError):
            call(**bad)
    for bad in (dict(mask=c.mask[:, :, :0]), dict(mask=c.mask.long()), dict(ctx_len=ctx.long()), dict(q=c.q.transpose(1, 2)),
                dict(lse=torch.empty((1, 4), device="cuda")), dict(q=c.q[..., :32]), dict(n_nodes=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(q=c.q.half())


def test_tensors_of_another_device_are_refused(monkeypatch):
    import dspark_draft_selection_gb300 as ds
    c = Q8Case(1, 1, 4, 2, 64, 16, [50], None).run()
    monkeypatch.setattr(ds._binding, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        c.run()
