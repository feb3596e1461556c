"""GPU parity of dspark_tree_mask and dspark_tree_accept against the oracle (whole numbers: equal)."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.gpu_util import dev, host

pytestmark = pytest.mark.gpu

EINVAL = 1


def random_trees(rng, R, T, back):
    parent = np.full((R, T), -1, np.int32)
    for r in range(R):
        for i in range(1, T):
            parent[r, i] = rng.integers(max(-1, i - back), i)
    return parent


def node_counts(rng, R, T):
    n = rng.integers(0, T + 1, R).astype(np.int32)
    n[0] = T
    return n


@pytest.mark.parametrize("T", [1, 2, 7, 31, 32, 33, 64, 65, 100, 128, 129, 256, 257, 511, 512])
@pytest.mark.parametrize("back", [1, 5, 1000])             # chains, trees, forests
def test_mask_and_positions(T, back):
    import dspark_draft_selection_gb300 as ds
    rng = np.random.default_rng(T * 7 + back)
    R = 3
    parent, n = random_trees(rng, R, T, back), node_counts(rng, R, T)
    base = rng.integers(0, 100000, R).astype(np.int32)
    mask, pos, st = ds.dspark_tree_mask(dev(parent), n_nodes=dev(n), base=dev(base))
    assert ds.read_status(st) == 0
    for r in range(R):
        sees, want = tree.tree_mask(parent[r], n[r], base[r])
        np.testing.assert_array_equal(host(mask[r]), tree.words(sees))
        np.testing.assert_array_equal(host(pos[r]), np.where(np.arange(T) < n[r], want, 0))


def test_mask_defaults_are_full_chains_at_zero():
    import dspark_draft_selection_gb300 as ds
    mask, pos, st = ds.dspark_tree_mask(None, R=2, T=70)
    assert ds.read_status(st) == 0
    sees, want = tree.tree_mask(np.arange(-1, 69), 70)
    for r in range(2):
        np.testing.assert_array_equal(host(mask[r]), tree.words(sees))
        np.testing.assert_array_equal(host(pos[r]), want)
    assert ds.dspark_tree_mask(torch.zeros((0, 4), dtype=torch.int32, device="cuda"))[0].shape == (0, 4, 1)


@pytest.mark.parametrize("bad", [3, 9, -2, 2 ** 31 - 1])
def test_a_parent_that_is_not_before_its_node_is_reported_and_makes_a_root(bad):
    import dspark_draft_selection_gb300 as ds
    parent = np.arange(-1, 7, dtype=np.int32)[None].copy()
    parent[0, 3] = bad
    mask, pos, st = ds.dspark_tree_mask(dev(parent))
    assert ds.read_status(st) == EINVAL
    sees, want = tree.tree_mask(parent[0], 8)
    np.testing.assert_array_equal(host(mask[0]), tree.words(sees))
    np.testing.assert_array_equal(host(pos[0]), want)
    for count in (-1, 9):
        mask, pos, st = ds.dspark_tree_mask(dev(parent), n_nodes=dev(np.array([count], np.int32)))
        assert ds.read_status(st) == EINVAL and not mask.any() and not pos.any()


@pytest.mark.parametrize("T", [1, 2, 16, 127, 128, 129, 512])
@pytest.mark.parametrize("words", [1, 3])                  # one token: every walk goes all the way down
def test_acceptance(T, words):
    import dspark_draft_selection_gb300 as ds
    rng = np.random.default_rng(T + words)
    R = 6
    parent, n = random_trees(rng, R, T, 3), node_counts(rng, R, T)
    n[1] = 0
    tokens, best = (rng.integers(0, words, (R, T)).astype(np.int32) for _ in range(2))
    out, acc, path, st = ds.dspark_tree_accept(dev(tokens), dev(parent), dev(best), n_nodes=dev(n))
    assert ds.read_status(st) == 0
    for r in range(R):
        o, a, p = tree.accept(tokens[r], parent[r], best[r], n[r])
        np.testing.assert_array_equal(host(out[r]), o)
        np.testing.assert_array_equal(host(path[r]), p)
        assert int(acc[r]) == a


def test_acceptance_of_chains_is_argmax_matching():
    import dspark_draft_selection_gb300 as ds
    rng = np.random.default_rng(9)
    tokens, best = (rng.integers(0, 2, (40, 8)).astype(np.int32) for _ in range(2))
    out, acc, path, st = ds.dspark_tree_accept(dev(tokens), None, dev(best))
    for r in range(40):
        a = 0
        while a + 1 < 8 and tokens[r, a + 1] == best[r, a]:
            a += 1
        assert int(acc[r]) == a and host(path[r])[a] == a and host(out[r])[a] == best[r, a]


def test_refusals_launch_nothing():
    import dspark_draft_selection_gb300 as ds
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ds.DsparkError):
        ds.dspark_tree_mask(z(1, 513))
    with pytest.raises(ds.DsparkError):
        ds.dspark_tree_accept(z(1, 513), None, z(1, 513))
    with pytest.raises(ValueError):
        ds.dspark_tree_mask(z(2, 8), n_nodes=z(3))
    with pytest.raises(ValueError):
        ds.dspark_tree_accept(z(2, 8), z(2, 8).long(), z(2, 8))
    with pytest.raises(ValueError):
        ds.dspark_tree_accept(z(2, 16)[:, ::2], None, z(2, 8))
