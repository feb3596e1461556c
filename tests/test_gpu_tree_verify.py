"""GPU parity of dspark_tree_verify against the float64 oracle: tokens, counts and paths are equal. (Sums of 48 bits against 64: a draw could
differ only where its target lies within about 2^-45 of a running sum.)"""
import numpy as np
import pytest
import torch

from oracle import q8
from tests.gpu_util import dev
from tests.test_gpu_tree import random_trees

pytestmark = pytest.mark.gpu

EINVAL, ERANGE, ENONFINITE = 1, 2, 5


class Trees:
    def __init__(self, seed, R, T, V, drawn, back=5, near=0.7, pad=0):
        self.rng = rng = np.random.default_rng(seed)
        self.R, self.T, self.V, self.drawn = R, T, V, drawn
        z = 2.0 * rng.standard_normal((R, T, V))
        soft = lambda x: (np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
        self.q = soft(z) if drawn else None
        self.p = soft(z + near * rng.standard_normal((R, T, V)))
        self.parent = random_trees(rng, R, T, back).astype(np.int32)
        self.tokens = np.zeros((R, T), np.int32)
        order = np.argsort(-z, -1)
        for r in range(R):
            for i in range(1, T):
                c = self.parent[r, i]
                if c < 0:
                    continue
                if drawn:
                    w = self.q[r, c].astype(np.float64)
                    self.tokens[r, i] = rng.choice(V, p=w / w.sum())
                else:
                    self.tokens[r, i] = order[r, c, min(V - 1, int((self.parent[r, :i] == c).sum()))]
        self.n = np.where(np.arange(R) % 3 == 2, rng.integers(0, T + 1, R), T).astype(np.int32)
        self.ua, self.ud = rng.random((R, T)), rng.random(R)
        self.pad = pad

    def rows(self, x):
        if x is None:
            return None
        t = torch.full((self.R, self.T, self.V + self.pad), float("nan"), device="cuda")
        t[..., :self.V] = dev(x)
        return t[..., :self.V]

    def run(self, **kw):
        import dspark_draft_selection_gb300 as ds
        got = ds.dspark_tree_verify(self.rows(self.p), dev(self.tokens), None if self.parent is None else dev(self.parent), dev(self.ua),
                                    dev(self.ud), q=self.rows(self.q), n_nodes=dev(self.n), **kw)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in got[:3]] + [ds.read_status(got[3])]

    def want(self):
        par = np.broadcast_to(np.arange(self.T) - 1, (self.R, self.T)) if self.parent is None else self.parent
        each = [q8.verify(self.p[r], None if self.q is None else self.q[r], self.tokens[r], par[r], int(self.n[r]), self.ua[r], self.ud[r])
                for r in range(self.R)]
        return [np.stack([e[k] for e in each]) for k in range(3)]

    def check(self, status=0):
        got = self.run()
        for g, w in zip(got, self.want()):
            np.testing.assert_array_equal(g, w)
        assert got[3] == status
        return self


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("R,T,V,pad", [(1, 1, 1, 0), (1, 2, 3, 0), (7, 9, 50, 0), (5, 16, 1001, 3), (3, 40, 4096, 4), (200, 5, 333, 0),
                                       (2, 12, 20011, 1), (700, 3, 64, 0)])
def test_trees(R, T, V, pad, drawn):
    Trees(R + T + V, R, T, V, drawn, pad=pad).check()


@pytest.mark.parametrize("total", [0.992, 1.008])
@pytest.mark.parametrize("V", [7, 3001])
def test_rows_that_were_rounded(V, total):
    """Rows that sum to 1 within 1/100 only, with proposals that have little in common with them, so that a residual keeps nearly all of a
    row's mass and many siblings are tested against it."""
    t = Trees(V, 40, 24, V, True, back=2, near=6.0)
    t.p = (t.p * np.float32(total)).astype(np.float32)
    t.check()


@pytest.mark.parametrize("drawn", [False, True])
def test_full_vocabulary(drawn):
    Trees(3, 2, 6, 151936, drawn).check()


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("T", [512, 130])
def test_stars_and_long_chains(drawn, T):
    """Every node a child of the first (refusal after refusal), the same token many times among them; and chains."""
    t = Trees(T, 3, T, 40, drawn, near=3.0)
    t.parent = np.zeros((3, T), np.int32)
    t.parent[:, 0] = -1
    t.ua = 0.5 + 0.5 * t.ua                                  # refused more often
    t.tokens[1] = 7
    t.n[:] = T
    t.check()
    t = Trees(T + 1, 3, T, 40, drawn, near=0.01)
    t.parent = None
    t.check()
    assert not drawn or (t.want()[1] > 3).any()              # drafted from nearly the target: deep walks


@pytest.mark.parametrize("drawn", [False, True])
def test_greedy_rows(drawn):
    """Rows of one certain id: what greedy acceptance gives."""
    t = Trees(5, 6, 10, 30, drawn)
    best = t.rng.integers(0, 3, (6, 10))
    t.tokens = t.rng.integers(0, 3, (6, 10)).astype(np.int32)
    t.p = np.eye(30, dtype=np.float32)[best]
    t.check()


def test_edges():
    t = Trees(6, 4, 5, 8, True)
    t.ud[:] = [0.0, 1.0 - 2.0 ** -53, 0.5, 0.25]
    t.p[1, :, 5:] = 0.0                                      # the last id above 0 is not the last
    t.p[2] = t.q[2]                                          # equal: nothing is refused
    t.ua[2] = 1.0 - 2.0 ** -53
    t.check()
    t.n[:] = [0, 5, 1, 5]
    t.check()
    t.tokens[3, 1:] = [-1, 8, 2 ** 31 - 1, 3]
    t.parent[3] = [-1, 0, 0, 0, 0]
    t.n[3] = 5
    t.check(ERANGE)


@pytest.mark.parametrize("drawn", [False, True])
def test_no_mass_left_and_rows_that_are_no_distribution(drawn):
    t = Trees(8, 4, 3, 16, drawn)
    t.parent[:] = [-1, 0, 0]
    t.n[:] = 3
    t.p[0, 0] = 0.0                                          # a certain id, refused through u: the residual is empty
    t.p[0, 0, 4] = 1.0
    t.tokens[0, 1:] = 4
    t.ua[0] = 1.0
    if drawn:
        t.q[0, 0] = t.p[0, 0]
    t.check()
    t.p[1, :] = 0.0
    t.p[2, :] = np.inf
    t.p[3, :, 3] = np.nan
    got = t.run()
    assert got[3] == ENONFINITE
    for r in range(1, 4):
        assert got[0][r][got[1][r]] == -1 and 0 <= got[1][r] < 3


def test_bad_parents_and_counts():
    t = Trees(9, 5, 6, 20, False)
    t.parent[0] = [-1, 5, 0, -7, 9, 2]                       # such nodes are never reached
    t.n[:] = [6, 7, -1, 6, 6]
    got = t.run()
    assert got[3] == EINVAL and got[1][1] == got[1][2] == -1 and (got[0][1] == -1).all() and (got[2][2] == -1).all()
    t.n[1:3] = 0
    fixed = t.parent.copy()
    fixed[0] = [-1, -1, 0, -1, -1, 2]
    t.parent = fixed
    for g, w in zip(got, t.want()):
        np.testing.assert_array_equal(g, w)


def test_streams_and_graphs():
    import dspark_draft_selection_gb300 as ds
    t = Trees(10, 9, 12, 5000, True)
    want = t.want()
    p, q, tok, par, ua, ud, n = t.rows(t.p), t.rows(t.q), dev(t.tokens), dev(t.parent), dev(t.ua), dev(t.ud), dev(t.n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ds.dspark_tree_verify(p, tok, par, ua, ud, q=q, n_nodes=n, stream=side)
    side.synchronize()
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)
    out, st = tuple(torch.empty_like(x) for x in got[:3]), ds.new_status()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds.dspark_tree_verify(p, tok, par, ua, ud, q=q, n_nodes=n, out=out, status=st)
    for k in range(3):
        for x in out:
            x.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        for y, w in zip(out, want):
            np.testing.assert_array_equal(y.cpu().numpy(), w)
