"""Pins of the oracle of the cache in 8 bits and of sampled acceptance along a tree (CPU)."""
import numpy as np
import pytest
import torch

from oracle import q8


@pytest.mark.parametrize("e4m3", [True, False])
def test_codes_are_the_nearest_numbers(e4m3):
    rng = np.random.default_rng(1)
    for k in range(60):
        y = (rng.standard_normal(32) * 10.0 ** rng.uniform(-30, 30)).astype(np.float32)
        codes, byte = q8.quantise_block(y, e4m3)
        e, most = int(byte) - 127, 448.0 if e4m3 else 127.0
        m = np.abs(y.astype(np.float64)).max()
        assert m <= most * 2.0 ** e and (e == -126 or m > most * 2.0 ** (e - 1))
        every = q8.E4M3[:127] if e4m3 else np.arange(128.0)
        got = q8.numbers(codes[None], np.array([[byte]], np.uint8), e4m3)[0]
        z = np.abs(y.astype(np.float64)) * 2.0 ** -e
        best = np.abs(z[:, None] - every[None]).min(1)
        np.testing.assert_array_equal(np.abs(np.abs(got) * 2.0 ** -e - z), best)
        assert np.all((got == 0) | (np.sign(got) == np.sign(y)))


def test_e4m3_is_torchs():
    z = np.concatenate([np.linspace(-448, 448, 30001), 2.0 ** np.linspace(-12, 8, 3001)]).astype(np.float32)
    t = torch.from_numpy(z).to(torch.float8_e4m3fn)
    for lo in range(0, len(z), 32):
        block = np.append(z[lo:lo + 31], np.float32(448))    # exponent 0
        codes, byte = q8.quantise_block(block, True)
        assert byte == 127
        np.testing.assert_array_equal(codes[:-1] & 127, t[lo:lo + 31].view(torch.uint8).numpy() & 127)
    np.testing.assert_array_equal(q8.E4M3[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("e4m3", [True, False])
def test_what_is_not_finite(e4m3):
    y = np.array([np.nan, np.inf, -np.inf, 1.0, -0.5] + [0.0] * 27, np.float32)
    codes, byte = q8.quantise_block(y, e4m3)
    got = q8.numbers(codes[None], np.array([[byte]], np.uint8), e4m3)[0]
    top = (448.0 if e4m3 else 127.0) * 2.0 ** (int(byte) - 127)
    assert list(got[:3]) == [0.0, top, -top] and abs(got[3] - 1.0) <= (2.0 ** -4 if e4m3 else 2.0 ** -7) and 1.0 <= top < 2.0


def _exact_rule(p, q, u):
    """The textbook steps with the residual normalised each time."""
    rho = p.copy()
    for x, ux in u:
        if ux < min(1.0, rho[x] / q[x]):
            return x, rho
        rho = np.maximum(rho - q, 0)
        rho /= rho.sum()
    return None, rho


def test_closed_form_of_the_residual():
    """a and b stand for one normalised residual after the other."""
    rng = np.random.default_rng(2)
    for k in range(50):
        p, q = rng.dirichlet(np.ones(9) * 0.5).astype(np.float32), rng.dirichlet(np.ones(9) * 0.5).astype(np.float32)
        p, q = p / p.sum(), q / q.sum()
        tokens = np.concatenate([[0], rng.choice(9, 4, p=q.astype(np.float64) / q.astype(np.float64).sum())])
        ua, ud = rng.random(5), rng.random()
        out, acc, path = q8.verify(np.stack([p] * 5), np.stack([q] * 5), tokens, np.array([-1, 0, 0, 0, 0]), 5, ua, ud)
        x, rho = _exact_rule(p.astype(np.float64), q.astype(np.float64), list(zip(tokens[1:], ua[1:])))
        if x is None:
            assert acc == 0 and out[0] == q8.pick(rho, ud)
        else:
            assert acc == 1 and out[0] == x


@pytest.mark.parametrize("drawn", [True, False])
def test_tokens_follow_the_target(drawn):
    """Whatever is drafted, the first token has the target's distribution (20,000 tries; a frequency is off by 5 sigma
    at most, 5 sqrt(0.25 / N))."""
    rng = np.random.default_rng(3)
    V, N = 4, 20000
    p, q = np.array([0.5, 0.2, 0.25, 0.05], np.float32), np.array([0.1, 0.6, 0.2, 0.1], np.float32)
    count = np.zeros(V)
    for _ in range(N):
        kids = rng.choice(V, 3, p=q.astype(np.float64) / q.astype(np.float64).sum()) if drawn else [1, 2, 1]
        out, acc, path = q8.verify(np.stack([p] * 4), np.stack([q] * 4) if drawn else None, np.array([0, *kids]), np.array([-1, 0, 0, 0]), 4,
                                   rng.random(4), rng.random())
        count[out[0]] += 1
    assert np.abs(count / N - p).max() < 5 * (0.25 / N) ** 0.5


def test_edges():
    p = np.array([[0.0, 1.0, 0.0], [0.25, 0.25, 0.5]], np.float32)
    assert q8.verify(p, p, np.array([0, 1]), np.array([-1, 0]), 0, np.zeros(2), 0.0)[1] == -1
    out, acc, path = q8.verify(p, p, np.array([0, 1]), np.array([-1, 0]), 2, np.array([0, 0.999]), 0.6)
    assert acc == 1 and list(out) == [1, 2] and list(path) == [0, 1]
    out, acc, _ = q8.verify(p, None, np.array([0, 2]), np.array([-1, 0]), 2, np.zeros(2), 0.999)   # certain of 2, which p excludes
    assert acc == 0 and out[0] == 1
    out, acc, _ = q8.verify(p, None, np.array([0, 7]), np.array([-1, 0]), 2, np.zeros(2), 0.5)     # no such id
    assert acc == 0 and out[0] == 1
