"""Pins of the oracle's tree functions against what the mathematics fixes (CPU only)."""
import numpy as np
import pytest

from oracle import tree


def _tree(rng, T):
    return np.array([-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, T)])


def test_mask_is_the_closure_of_the_parent_matrix():
    rng = np.random.default_rng(1)
    for T in (1, 2, 9, 40):
        parent = _tree(rng, T)
        P = np.eye(T, dtype=np.int64)
        for i, p in enumerate(parent):
            if p >= 0:
                P[i, p] = 1
        sees, pos = tree.tree_mask(parent, T, 7)
        np.testing.assert_array_equal(sees, np.linalg.matrix_power(P, T).astype(bool) if T < 20 else _power(P, T))
        np.testing.assert_array_equal(pos, 7 + sees.sum(1) - 1)
        w = tree.words(sees).view(np.uint32)
        for i in range(T):
            assert sum(int(x) << (32 * k) for k, x in enumerate(w[i])) == sum(1 << j for j in range(T) if sees[i, j])


def _power(P, T):
    x = P.astype(bool)
    for _ in range(T):
        x = (x.astype(np.int64) @ P) > 0
    return x


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations_keep_lengths_and_compose_by_difference(interleaved):
    rng = np.random.default_rng(2)
    h, D = 6, 16
    f = 100.0 ** (-np.arange(h) / h)
    q, k = rng.standard_normal(D), rng.standard_normal(D)
    turn = lambda x, p: tree.rope(x, np.cos(p * f), np.sin(p * f), interleaved)  # noqa: E731
    np.testing.assert_allclose(turn(turn(q, 3.0), 5.0), turn(q, 8.0), atol=1e-12)
    np.testing.assert_allclose(turn(q, 9.0) @ turn(k, 4.0), turn(q, 5.0) @ k, atol=1e-12)
    np.testing.assert_array_equal(turn(q, 0.0), q)
    np.testing.assert_array_equal(turn(q, 2.0)[2 * h:], q[2 * h:])
    np.testing.assert_allclose(np.linalg.norm(turn(q, 7.0)), np.linalg.norm(q))


def test_a_node_is_the_last_token_of_its_chain():
    rng = np.random.default_rng(3)
    T, S, Hq, H, D = 11, 9, 4, 2, 8
    parent = _tree(rng, T)
    q, k, v = rng.standard_normal((T, Hq, D)), rng.standard_normal((S + T, H, D)), rng.standard_normal((S + T, H, D))
    sees, _ = tree.tree_mask(parent, T)
    out, lse, mag, _ = tree.attention(q, k, v, np.concatenate([np.ones((T, S), bool), sees], 1), 0.4, 3.0)
    for i in range(T):
        chain = []
        c = i
        while c >= 0:
            chain.append(c)
            c = parent[c]
        at = list(range(S)) + [S + c for c in reversed(chain)]
        for hq in range(Hq):
            x = 3.0 * np.tanh(0.4 * (k[at, hq // 2] @ q[i, hq]) / 3.0)
            w = np.exp(x) / np.exp(x).sum()
            np.testing.assert_allclose(out[i, hq], w @ v[at, hq // 2], rtol=1e-12)
            np.testing.assert_allclose(lse[i, hq], np.log(np.exp(x).sum()), rtol=1e-12)
    assert np.all(mag >= np.abs(out) - 1e-15)


def test_a_wide_cap_is_no_cap_and_an_empty_row_is_zero():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    sees = np.ones((3, 5), bool)
    sees[1] = False
    k[0] = np.inf                                        # not seen by row 2
    sees[2, 0] = False
    sees[0, 0] = False
    a, la, _, _ = tree.attention(q, k, v, sees, 0.3)
    b, lb, _, _ = tree.attention(q, k, v, sees, 0.3, 1e6)
    np.testing.assert_allclose(a, b, rtol=1e-9)
    assert np.all(a[1] == 0) and np.all(la[1] == -np.inf) and np.all(np.isfinite(a))


def test_acceptance_is_the_longest_agreeing_path():
    rng = np.random.default_rng(5)
    for _ in range(200):
        T = int(rng.integers(1, 14))
        parent, tokens, best = _tree(rng, T), rng.integers(0, 3, T), rng.integers(0, 3, T)
        out, acc, path = tree.accept(tokens, parent, best, T)
        assert path[0] == 0 and list(path[:acc + 1]) == sorted(path[:acc + 1])
        agree = {0}
        for i in range(1, T):                            # the first of several equal siblings counts
            twin = any(parent[j] == parent[i] and tokens[j] == tokens[i] for j in range(1, i))
            if parent[i] in agree and tokens[i] == best[parent[i]] and not twin:
                agree.add(i)
        assert set(path[:acc + 1]) == agree
        assert list(out[:acc]) == [tokens[i] for i in path[1:acc + 1]] and out[acc] == best[path[acc]]
        assert np.all(out[acc + 1:] == -1) and np.all(path[acc + 1:] == -1)


def test_commit_moves_rows_to_the_front():
    rows = np.arange(12.0)
    got = tree.commit(rows, 3, [0, 2, 5, -1], 2)
    np.testing.assert_array_equal(got, [0, 1, 2, 3, 5, 8, 6, 7, 8, 9, 10, 11])
