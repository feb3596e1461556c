"""Attention over codes where whole blocks of 32 columns are zeros, which the quantising append writes under the least power of two
(padded head columns, keys or values that vanish), and where the powers of one slice of keys lie far apart.

Tolerances as in tests/test_gpu_tree_attention.py. The kernel for few rows a key head rounds weights to f16: half a step, 2^-11 of a weight, instead of bf16's
2^-8, down to f16's least normal number; below it by at most 2^-25, against a largest weight of at least 2^7, so by 2^-32 of the row's largest weight."""
import numpy as np
import pytest
import torch

from oracle import tree
from tests.test_gpu_cache import f64, slots_of
from tests.test_gpu_q8_attention import Q8Case
from tests.test_gpu_q8_cache import numbers

pytestmark = pytest.mark.gpu


def zero(c, which, blocks, step, byte=1, minus=False):
    """Blocks of keys (0) or values (1) of every `step`-th slot become zeros, with a scale byte that means the least power."""
    codes, scale = c.cache[which].view(torch.uint8), c.cache[2 + which]
    for r in range(c.R):
        s = torch.arange(0, c.ctx[r] + c.n[r], step, device="cuda")
        at = c.table[r].long()[s // c.page], s % c.page
        for b in blocks:
            x = codes[at]
            x[..., 32 * b:32 * b + 32] = 128 if minus else 0
            codes[at] = x
            y = scale[at]
            y[..., b] = byte
            scale[at] = y
    c.k, c.v = numbers(c.cache, c.code)
    return c


def check_f16(c):
    """As Case.check, with weights of f16's precision."""
    assert int(c.status) == 0
    worst = 0.0
    for r in range(c.R):
        end = c.ctx[r] + c.n[r]
        sees = np.concatenate([np.ones((c.T, c.ctx[r]), bool), c.sees[r][:, :c.n[r]]], 1)
        k, v = (f64(slots_of(x, c.table, r, end)) for x in (c.k, c.v))
        want, _, mag, big = tree.attention(f64(c.q[r]), k, v, sees, c.scale)
        eps = 2 * (c.D + 8) * 2.0 ** -24 * big + 2.0 ** -20 + end * 2.0 ** -24
        tol = (eps[..., None] + 2.0 ** -11 * (1 + 2.0 ** -7)) * mag + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want) + end * 2.0 ** -32 * np.abs(v).max() + 1e-30
        worst = max(worst, (np.abs(f64(c.out[r]) - want) / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq", [(1, 8), (4, 8), (8, 8)])         # 4, 16 and 32 rows a key head
@pytest.mark.parametrize("which", ["none", "keys", "values", "both"])
@pytest.mark.parametrize("step", [1, 5])                           # of every slot, or of some slots of every slice
def test_blocks_of_zeros_keep_the_weights_precision(code, D, T, Hq, which, step):
    c = Q8Case(T + D, T, Hq, 2, D, 16, [3, 19, 60, 2], None, "bf16", code, mask="chain", scale=0.3 * D ** -0.5)
    last = D // 32 - 1
    if which in ("keys", "both"):
        zero(c, 0, [last], step, byte=1 if step == 1 else 0)
    if which in ("values", "both"):
        zero(c, 1, [0, last], step, minus=code == "e4m3")
    check_f16(c.run())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [32, 64, 80, 128])
@pytest.mark.parametrize("dtype,T,Hq", [("bf16", 1, 2), ("bf16", 9, 6), ("bf16", 40, 4), ("bf16", 90, 8), ("f32", 5, 4)])
def test_blocks_of_zeros_in_every_kernel(code, D, dtype, T, Hq):
    """All keys' or values' blocks of some slots, single blocks of others, and a request that holds nothing but zeros."""
    c = Q8Case(T + D, T, Hq, 2, D, 16, [70, 0, 200, 33], None, dtype, code)
    nb = (D + 31) // 32
    zero(c, 0, range(nb), 7)
    zero(c, 1, range(nb), 11)
    zero(c, 0, [nb - 1], 3)
    zero(c, 1, [0], 2)
    c.run().check()
    zero(c, 0, range(nb), 1)
    zero(c, 1, range(nb), 1)
    c.run().check()
    assert (c.out == 0).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("T,Hq", [(1, 8), (4, 8), (8, 8), (40, 4)])
@pytest.mark.parametrize("low,high", [(95, 117), (1, 117), (113, 117)])
def test_powers_of_keys_far_apart_within_a_slice(code, D, T, Hq, low, high):
    """Keys whose blocks' powers differ by more than an f16 factor reaches, blocks of zeros among them; and, in the last case, by less."""
    c = Q8Case(T + D, T, Hq, 2, D, 16, [5, 130, 48], None, "bf16", code, mask="chain")
    k = c.cache[2]
    k.copy_(torch.randint(low, high + 1, k.shape, generator=c.gen).to(torch.uint8))
    zero(c, 0, [1], 4).run().check()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("byte", [0, 1, 2])
@pytest.mark.parametrize("T", [1, 6])
def test_the_least_power_of_blocks_that_are_not_zeros(code, byte, T):
    """Values under the least powers beside blocks of zeros under the same byte: what they stand for, not nothing. The largest of them is 448 * 2^-125."""
    c = Q8Case(T, T, 4, 2, 128, 16, [37], None, "bf16", code, mask="chain")
    c.cache[3].fill_(byte)
    zero(c, 1, [2], 3, byte).run()
    end = 37 + T
    k, v = (f64(slots_of(x, c.table, 0, end)) for x in (c.k, c.v))
    want, _, mag, big = tree.attention(f64(c.q[0]), k, v, np.concatenate([np.ones((T, 37), bool), np.tri(T, dtype=bool)], 1), c.scale)
    eps = 2 * 136 * 2.0 ** -24 * big + 2.0 ** -20 + end * 2.0 ** -24
    # columns below 2^-126 may be read as 0
    tol = (eps[..., None] + 2.0 ** -8 * (1 + 2.0 ** -7)) * mag + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want) + 2.0 ** -126
    assert int(c.status) == 0 and (np.abs(f64(c.out[0]) - want) <= tol).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("T,Hq", [(1, 8), (4, 8), (8, 8), (40, 4)])
@pytest.mark.parametrize("large", [1.0, 2.0 ** 12, 2.0 ** 26])
def test_queries_of_a_wide_range(code, T, Hq, large):
    """A block of query columns far above the others, where keys are zeros. With few rows a key head a query column is taken to within 2^-38 of its row's
    largest, so a score is off by that times the sum of scale |k|, and a weight by the exponential of twice that (its own and the sum's)."""
    c = Q8Case(T, T, Hq, 2, 128, 16, [21, 60], None, "bf16", code, mask="chain", scale=0.05)
    q = c.q.clone()
    q[..., 32:64] *= large
    c.q = q
    zero(c, 0, [1], 1).run()
    for r in range(c.R):
        end = c.ctx[r] + T
        k, v = (f64(slots_of(x, c.table, r, end)) for x in (c.k, c.v))
        x = f64(q[r])
        want, _, mag, big = tree.attention(x, k, v, np.concatenate([np.ones((T, c.ctx[r]), bool), np.tri(T, dtype=bool)], 1), c.scale)
        off = 2.0 ** -38 * c.scale * np.abs(x).max(-1) * np.abs(k).sum(-1).max() if T * Hq // 2 <= 32 else 0.0
        eps = 2 * 136 * 2.0 ** -24 * big + 2.0 ** -20 + end * 2.0 ** -24 + np.expm1(2 * off)
        tol = (eps[..., None] + 2.0 ** -8 * (1 + 2.0 ** -7)) * mag + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(want) + 1e-30
        assert int(c.status) == 0 and (np.abs(f64(c.out[r]) - want) <= tol).all()
