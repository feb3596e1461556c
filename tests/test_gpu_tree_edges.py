"""Edges of dspark_tree_attention. Tolerances as in test_gpu_tree_attention.py; a cap's own
error is 2^-20 of the smaller of the cap and the scores' magnitude (a score's rounding is relative to itself)."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.test_gpu_cache import f64, slots_of
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


def place(c, r, j):
    """Index of slot j of request r in the cache."""
    return int(c.table[r, j // c.page]), j % c.page


def against_oracle(c, requests, rows=None, status=0):
    """Every element of the result, infinities with their sign and what is not a number included."""
    assert int(c.status) == status
    for r in requests:
        ctx, n = c.ctx[r], c.n[r]
        i = np.arange(c.T) if rows is None else np.array(rows)
        sees = np.concatenate([np.ones((c.T, ctx), bool), c.sees[r][:, :n]], 1)
        sees[n:] = False
        k, v = (f64(slots_of(x, c.table, r, ctx + n)) for x in (c.k, c.v))
        with np.errstate(invalid="ignore"):
            want, lse, mag, big = tree.attention(f64(c.q[r])[i], k, v, sees[i], c.scale, c.softcap)
        eps = 2 * (c.D + 8) * 2.0 ** -24 * big + 2.0 ** -20 + (ctx + n) * 2.0 ** -24 + 2.0 ** -20 * np.minimum(c.softcap, big)
        half = 2.0 ** -8 * (1 + 2.0 ** -7) if c.dtype == "bf16" else 0.0
        got, got_lse = f64(c.out[r])[i], f64(c.lse[r])[i]
        fin = np.isfinite(want)
        np.testing.assert_array_equal(got[~fin], want[~fin])
        with np.errstate(invalid="ignore"):
            tol, off = (eps[..., None] + half) * mag + half * np.abs(want) + 1e-30, np.abs(got - want)
        bad = ~(off[fin] <= tol[fin])
        assert not bad.any(), (r, int(bad.sum()), (off[fin] / tol[fin]).max())
        ok = np.isfinite(lse)
        np.testing.assert_array_equal(got_lse[~ok], lse[~ok])
        assert np.all(np.abs(got_lse[ok] - lse[ok]) <= (eps + 2.0 ** -22 * (1 + np.abs(lse)))[ok])


# --- a wait that ran out ---
@pytest.mark.parametrize("R,ctx,T", [(30, 100, 8), (60, 100, 8), (60, 200, 8), (20, 150, 80), (60, 900, 80)])
def test_a_wait_that_ran_out_leaves_nothing_in_flight(R, ctx, T):
    """Blocks with short shares have every copy under way when their first wait runs out. The calls right behind them, whose
    blocks get the same shared memory, are as ever."""
    import dspark_draft_selection_gb300 as ds
    c = Case(13, T, 4, 2, 128, 16, [ctx] * R, None, mask="chain")
    c.run()
    want, want_lse = c.out.clone(), c.lse.clone()
    lens = torch.tensor(c.ctx, dtype=torch.int32, device="cuda")
    ws, out = ds.workspace(ds.OP_TREE_ATTENTION, R, T, 4 * 128, 2), torch.empty_like(c.out)
    for _ in range(20):
        late, good = ds.new_status(), ds.new_status()
        try:
            ds.dspark_test_set_first_wait_polls(0)
            ds.dspark_tree_attention(c.q, c.k, c.v, c.table, lens, scale=c.scale, out=out, ws=ws, status=late)
        finally:
            ds.dspark_test_set_first_wait_polls(0xFFFFFFFF)
        _, lse, _ = ds.dspark_tree_attention(c.q, c.k, c.v, c.table, lens, scale=c.scale, out=out, ws=ws, status=good)
        assert int(late) == 6 and int(good) == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


# --- values that are not finite ---
SIZES = [(8, 8), (40, 16)]                                   # T, query heads on two key heads: one tile of rows, two


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq", SIZES)
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_nodes_with_values_that_are_not_finite_behind_thousands_of_keys(dtype, T, Hq, softcap):
    """Rows that see such a node get what the sum gives in its columns, the others and the other columns are as
    without it: several nodes, both infinities in one column, one node in the last place."""
    c = Case(T, T, Hq, 2, 128, 16, [3001, 130], [T, T - 1], dtype, softcap=softcap)
    for r in range(2):
        last = c.n[r] - 1
        for j, h, col, x in ((1, 0, 5, float("inf")), (2, 0, 5, -float("inf")), (2, 1, 77, float("nan")), (4, 1, 0, float("inf")),
                             (last, 0, 127, -float("inf")), (last, 1, 64, float("nan"))):
            c.v[place(c, r, c.ctx[r] + j)][h, col] = x
    rows = None if T < 10 else [0, 1, 2, 3, 4, 5, 17, T - 2, T - 1]
    c.run()
    against_oracle(c, (0, 1), rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq", SIZES)
def test_committed_values_that_are_not_finite_reach_every_row(dtype, T, Hq):
    c = Case(T, T, Hq, 2, 64, 16, [1030, 20], None, dtype)
    for j, h, col, x in ((3, 0, 9, float("inf")), (1029, 1, 8, float("nan")), (1028, 0, 8, -float("inf"))):
        c.v[place(c, 0, j)][h, col] = x
    c.v[place(c, 0, 1030 + 2)][0, 9] = -float("inf")         # and a node against the committed infinity
    c.run()
    against_oracle(c, (0, 1), None if T < 10 else [0, 1, 2, 3, 9, T - 1])


def test_every_node_with_values_that_are_not_finite():
    """The widest tree, every value of it: rows whose mask holds nothing keep their committed mean."""
    c = Case(7, 512, 2, 1, 64, 16, [700], None, mask="any")
    for j in range(512):
        c.v[place(c, 0, 700 + j)] = float("nan") if j % 2 else float("inf")
    c.run()
    against_oracle(c, (0,), [0, 1, 2, 3, 4, 250, 252, 510, 511])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq", SIZES)
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_nodes_with_keys_and_values_that_are_not_finite(dtype, T, Hq, softcap):
    """An infinity in a node's key makes scores of both signs: a weight of 0 (none under a cap) times an infinite value is not
    a number, and the score of +inf spoils its row."""
    c = Case(T + 1, T, Hq, 2, 64, 16, [300, 0], [T, T - 1], dtype, softcap=softcap)
    for r, j, col, key, value in ((0, 1, 5, float("inf"), float("inf")), (0, 4, 9, -float("inf"), float("nan")),
                                  (1, 3, 5, -float("inf"), -float("inf")), (1, 2, 0, float("inf"), 1.0)):
        at = place(c, r, c.ctx[r] + j)
        c.k[at][:, col], c.v[at][:, 2 * col + 3] = key, value
    c.run()
    against_oracle(c, (0, 1), None if T < 10 else list(range(12)) + [T - 2, T - 1])


def times(T, Hq, bad, R=80, ctx=2000):
    """(best time of a clean call, of one with `bad` done to the case, the two results) of requests whose items have one block each."""
    import dspark_draft_selection_gb300 as ds
    c = Case(3, T, Hq, 2, 64, 16, [ctx] * R, None, mask="chain")
    lens = torch.tensor(c.ctx, dtype=torch.int32, device="cuda")
    ws, st, out = ds.workspace(ds.OP_TREE_ATTENTION, R, T, Hq * 64, 2), ds.new_status(), torch.empty_like(c.q)

    def took():
        best = 1e9
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            ds.dspark_tree_attention(c.q, c.k, c.v, c.table, lens, out=out, ws=ws, status=st)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    clean, good = took(), out.clone()
    bad(c)
    got = took()
    assert int(st) == 0
    return clean, got, good, out


@pytest.mark.parametrize("T,Hq", [(8, 8), (64, 8)])
@pytest.mark.parametrize("where", ["committed", "node"])
def test_a_value_that_is_not_finite_takes_no_longer(T, Hq, where):
    """One bad value in one request of many: the call's time is a clean call's (three times as much at most, for the
    clocks' sake)."""
    def bad(c):
        c.v[place(c, 41, 700 if where == "committed" else 2001)] = float("nan")

    clean, got, good, out = times(T, Hq, bad)
    assert torch.isnan(out[41].float()).any() and torch.equal(out[:41], good[:41]) and torch.equal(out[42:], good[42:])
    assert got < 3 * clean, (got, clean)


def test_a_tree_of_values_that_are_not_finite_takes_little_longer():
    """All 64 nodes of one request, each of which up to 64 rows see (as a model that broke down leaves them)."""
    def bad(c):
        for j in range(2000, 2064):
            c.v[place(c, 41, j)] = float("nan")

    clean, got, good, out = times(64, 8, bad)
    assert torch.isnan(out[41].float()).all() and torch.equal(out[:41], good[:41]) and torch.equal(out[42:], good[42:])
    assert got < 5 * clean, (got, clean)


# --- what is not seen ---
def same_bits_whatever_is_not_seen(dtype, softcap, T, Hq):
    """Keys past the end, keys of nodes that a row does not see and other rows' queries: ordinary ones, large ones or
    nothing sensible, the row's bits are the same."""
    c = Case(12, T, Hq, 2, 64, 16, [333, 20], [T, T - 3], dtype, softcap=softcap)
    c.run()
    assert int(c.status) == 0
    out, lse = c.out.clone(), c.lse.clone()
    used = torch.zeros(c.k.shape[:2], dtype=torch.bool, device="cuda")
    for r in range(2):
        for j in range(c.ctx[r] + c.n[r]):
            used[place(c, r, j)] = True
    for junk in (0.0, 60.0, 3e38, float("inf"), float("nan")):
        c.k[~used], c.v[~used] = junk, junk
        c.run()
        assert int(c.status) == 0 and torch.equal(c.out, out) and torch.equal(c.lse, lse), junk
    node = 2
    blind = [i for i in range(T) if not c.sees[0, i, node]]
    assert blind and not c.sees[0, blind[-1], node]
    at = place(c, 0, c.ctx[0] + node)
    keep = c.k[at].clone(), c.v[at].clone(), c.q[0, node].clone()
    for junk in (0.0, 60.0, 3e38, float("inf"), float("nan")):
        c.k[at], c.v[at], c.q[0, node] = junk, junk, junk
        c.run()
        assert int(c.status) == 0, junk
        assert torch.equal(c.out[0, blind], out[0, blind]) and torch.equal(c.lse[0, blind], lse[0, blind]), junk
        assert torch.equal(c.out[1], out[1])
    c.k[at], c.v[at], c.q[0, node] = keep


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq", [(9, 4), (70, 4)])
def test_what_is_not_seen_changes_no_bit(dtype, T, Hq):
    same_bits_whatever_is_not_seen(dtype, 0.0, T, Hq)


# --- the range of values ---
def along(c, r, h, scores):
    """Keys of request r, key head h, whose scores with every query (all of them made alike) are as given."""
    D = c.D
    unit = torch.ones(D, device="cuda")
    unit[::3] = -1.0
    c.q[r] = unit.to(c.q.dtype)
    s = torch.arange(len(scores), device="cuda")
    at = c.table[r].long()[s // c.page], s % c.page
    k = torch.tensor(scores, dtype=torch.float64, device="cuda")[:, None] / (D * c.scale) * unit
    c.k[at[0], at[1], h] = k.to(c.k.dtype)
    return at


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 70])                       # one tile of rows, two
@pytest.mark.parametrize("softcap", [20.0, 38.0, 50.0, 55.0])
def test_scores_that_reach_the_cap_late_with_large_values(dtype, T, softcap):
    """Hundreds of keys a little below zero, then some at the cap, in items that one block holds whole: whatever the reference
    was, finite values stay finite."""
    R = 90
    c = Case(5, T, 4, 2, 64, 16, [900] * R, None, dtype, mask="chain", scale=0.125, softcap=softcap)
    scores = np.full(900, -12.0)
    scores[[300, 301, 700, 899]] = 3000.0
    for r in (0, 8, 89):
        for h in range(2):
            along(c, r, h, scores)
    c.v *= 2.0 ** 60
    c.run()
    against_oracle(c, (0, 8, 89), None if T < 10 else [0, 1, 35, T - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
def test_rows_that_see_a_value_near_the_types_largest(dtype, T, softcap):
    """Maxima that rise by a few units behind the first tiles of items that one block holds whole, and a value of 3e38 on a
    key at the top."""
    R = 90
    c = Case(6, T, 4, 2, 64, 16, [500] * R, None, dtype, mask="chain", scale=0.125, softcap=softcap)
    scores = np.concatenate([np.linspace(-2, 0, 256), np.linspace(0, 4.5, 244)])
    for r in (0, 7, 89):
        for h in range(2):
            at = along(c, r, h, scores)
            c.v[int(at[0][497]), int(at[1][497]), h, 3:7] = 3e38
    c.run()
    against_oracle(c, (0, 7, 89), None if T < 10 else [0, 1, 35, T - 1])


# --- caps far from the scores ---
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 70])
@pytest.mark.parametrize("softcap", [1e-3, 0.3, 1e3, 1e5, 1e7, 1e10, 1e20, 3e38])
def test_caps_far_from_the_scores(dtype, T, softcap):
    """A cap far above the scores is no cap; one far below them leaves the signs."""
    c = Case(11, T, 4, 2, 64, 16, [600, 31], None, dtype, softcap=softcap).run()
    against_oracle(c, (0, 1), None if T < 10 else [0, 1, 35, T - 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [4.0, 30.0, 1e6])
@pytest.mark.parametrize("T,Hq", [(9, 4), (70, 4)])
def test_what_is_not_seen_changes_no_bit_under_a_cap(dtype, softcap, T, Hq):
    same_bits_whatever_is_not_seen(dtype, softcap, T, Hq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [1e-45, 1e-38, 1e-20, 1e-7, 1e-3])
def test_scores_of_nothing_under_tiny_caps(dtype, softcap):
    """Queries of zeros and keys of zeros beside others: every score is the cap, its negative or 0, the mean is the plain one."""
    c = Case(14, 6, 4, 2, 64, 16, [300, 0], None, dtype, softcap=softcap)
    c.q[0, 1], c.q[1, 0], c.q[0, 3, 1] = 0.0, 0.0, 0.0
    c.k[place(c, 0, 7)], c.k[place(c, 1, 2)] = 0.0, 0.0
    c.run()
    against_oracle(c, (0, 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [0.5, 30.0, 300.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("top", [0.01, 0.2, 0.36, 0.7, 0.97, 3.0])
def test_scores_up_to_and_past_the_cap(dtype, softcap, top):
    """The largest score at a share of the cap, others from as far below zero: every form of the cap up to its end."""
    c = Case(15, 3, 4, 2, 64, 16, [300], None, dtype, mask="chain", scale=0.125, softcap=softcap)
    for h in range(2):
        along(c, 0, h, np.linspace(-top, top, 300) * softcap)
    c.run()
    against_oracle(c, (0,))


# --- many requests, slots without a place ---
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,T,Hq,H,D", [(63, 3, 2, 1, 64), (64, 3, 2, 1, 64), (65, 3, 4, 2, 64), (200, 2, 4, 2, 128), (1024, 2, 2, 1, 64)])
def test_many_requests(dtype, R, T, Hq, H, D):
    """Ragged lengths, empty requests at the ends and among the others, up to the most requests of a call."""
    rng = np.random.default_rng(R)
    ctx, n = rng.integers(0, 300, R), rng.integers(0, T + 1, R)
    ctx[rng.random(R) < 0.2], n[rng.random(R) < 0.2] = 0, 0
    ctx[[0, R - 1]], n[[0, R - 1]] = 0, 0
    c = Case(R, T, Hq, H, D, 16, ctx.tolist(), n.tolist(), dtype).run()
    against_oracle(c, range(R))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_out_of_range_read_as_zeros(dtype):
    """Keys and values of such slots, committed or a node's, are zeros: scores of 0, nothing added."""
    c = Case(2, 6, 4, 2, 64, 16, [100, 40], None, dtype)
    table, pages = c.table.clone(), c.k.shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        for page, whole in ((2, 0), (6, 0), (0, 1)):         # slots 32..47 and the nodes' of request 0, the first of request 1
            c.table[whole, page] = bad
            c.run()
            assert int(c.status) == 2
            c.table.copy_(table)
            at = int(table[whole, page])
            kept = c.k[at].clone(), c.v[at].clone()
            c.k[at], c.v[at] = 0, 0                          # what the oracle reads there
            against_oracle(c, (0, 1), status=2)
            c.k[at], c.v[at] = kept


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slots_past_the_tables_row_are_left_out(dtype):
    """Committed slots past it are not seen, nodes there give zeros and -inf, the nodes before them do not see those."""
    c = Case(3, 6, 4, 2, 64, 16, [90, 40], None, dtype, mask="block")
    places = c.table.shape[1] * 16
    good = c.run().out.clone()
    for ctx, left in ((places - 6, 6), (places - 4, 4), (places, 0), (places + 5, 0), (10 ** 9, 0), (2 ** 31 - 1, 0)):
        c.ctx = [ctx, 40]
        c.run()
        c.ctx, c.n = [min(ctx, places), 40], [left, 6]
        against_oracle(c, (0, 1), status=0 if left == 6 else 2)
        assert torch.equal(c.out[1], good[1]) and not c.out[0, left:].any() and torch.all(c.lse[0, left:] == -float("inf"))
        c.n = [6, 6]
