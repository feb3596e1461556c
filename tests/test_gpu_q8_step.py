"""The operators of a tree's step over a cache in 8 bits together, as a server runs them: quantising append, attention, sampled acceptance,
commit and read back, several steps on one cache; each result against the oracle, from what the cache holds."""
import numpy as np
import pytest
import torch

from oracle import q8, tree
from tests.gpu_util import dev
from tests.test_gpu_tree import random_trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_steps_of_sampled_trees(code, captured):
    import dspark_draft_selection_gb300 as ds
    R, T, Hq, H, D, V, page, layers, per = 3, 9, 8, 2, 64, 50, 16, 2, 6
    rng = np.random.default_rng(1)
    cache = ds.q8_cache(R * per, page, H, D, layers=layers, dtype=code)
    layer = [tuple(c[i] for c in cache) for i in range(layers)]
    table = torch.randperm(R * per).int().reshape(R, per).cuda()
    h = D // 2
    ang = np.arange(200)[:, None] * 50.0 ** (-np.arange(h) / h)
    cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    cs, status = dev(cos_sin), ds.new_status()
    length = torch.zeros(R, dtype=torch.int32, device="cuda")
    ws = ds.workspace(ds.OP_TREE_ATTENTION_Q8, R, T, Hq * D, H)
    # everything that changes from step to step, at fixed places
    qkv = [torch.empty((R, T, Hq + 2 * H, D), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    parent, tokens = (torch.empty((R, T), dtype=torch.int32, device="cuda") for _ in range(2))
    p, q = (torch.empty((R, T, V), device="cuda") for _ in range(2))
    ua, ud = torch.empty((R, T), dtype=torch.float64, device="cuda"), torch.empty((R,), dtype=torch.float64, device="cuda")

    def step():
        mask, pos, _ = ds.dspark_tree_mask(parent, base=length, status=status)
        turned, outs = [], []
        for i in range(layers):
            x, k, v = qkv[i][:, :, :Hq], qkv[i][:, :, Hq:Hq + H], qkv[i][:, :, Hq + H:]
            x, _ = ds.dspark_rope_append_q8(x, k, v, pos, cs, layer[i], table, length, status=status)
            turned.append(x)
            outs.append(ds.dspark_tree_attention_q8(x, layer[i], table, length, mask=mask, ws=ws, status=status)[0])
        new, n, path, _ = ds.dspark_tree_verify(p, tokens, parent, ua, ud, q=q, status=status)
        read = [ds.dspark_cache_read_q8(layer[i], table, length + T, S=per * page, dtype=torch.float32, status=status)[:2] for i in range(layers)]
        grown, _ = ds.dspark_cache_commit_q8(cache, table, length, path, n, status=status)
        after = [ds.dspark_cache_read_q8(layer[i], table, grown, S=per * page, dtype=torch.float32, status=status)[:2] for i in range(layers)]
        return turned, outs, new, n, path, read, grown, after

    def fill():
        z = rng.standard_normal((R, T, V))
        soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
        par = np.minimum(random_trees(rng, R, T, 3), np.arange(T) - 1).astype(np.int32)
        par[:, 1:] = np.maximum(par[:, 1:], 0)
        for t in qkv:
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape)).to(torch.bfloat16))
        parent.copy_(torch.from_numpy(par))
        tokens.copy_(torch.from_numpy(rng.integers(0, 8, (R, T))).int())
        q.copy_(torch.from_numpy(soft(z)))
        p.copy_(torch.from_numpy(soft(z + 0.3 * rng.standard_normal(z.shape))))
        ua.copy_(torch.from_numpy(0.6 * rng.random((R, T))))
        ud.copy_(torch.from_numpy(rng.random(R)))

    graph = out = None
    if captured:
        fill()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
    for _ in range(4):
        fill()
        before = length.tolist()
        if captured:
            graph.replay()
        else:
            out = step()
        torch.cuda.synchronize()
        turned, outs, new, n, path, read, grown, after = out
        assert ds.read_status(status) == 0
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        for r in range(R):
            par = parent[r].tolist()
            sees, pos = tree.tree_mask(par, T, before[r])
            want = q8.verify(p[r].cpu().numpy(), q[r].cpu().numpy(), tokens[r].tolist(), par, T, ua[r].tolist(), float(ud[r]))
            for got, w in zip((new[r], n[r], path[r]), want):
                np.testing.assert_array_equal(got.cpu().numpy(), w)
            see = np.concatenate([np.ones((T, before[r]), bool), sees], 1)
            for i in range(layers):
                k, v = (f(x[r])[:before[r] + T] for x in read[i])
                codes, scale = q8.quantise(q8.turn(qkv[i][r, 0, Hq:Hq + H].float().cpu().numpy(), cos_sin[pos[0], :h], cos_sin[pos[0], h:], False),
                                           code is torch.float8_e4m3fn)
                np.testing.assert_array_equal(k[before[r]], q8.numbers(codes, scale, code is torch.float8_e4m3fn))
                x, _, mag, _ = tree.attention(f(turned[i][r]), k, v, see, D ** -0.5)
                # a rounding of each weight and one of the result, 2^-8 each at most, and float32 sums
                assert np.all(np.abs(f(outs[i][r]) - x) <= 2.0 ** -8 * (1 + 2.0 ** -6) * (mag + np.abs(x)) + 1e-6)
                kept = before[r] + int(n[r]) + 1
                for x, y in zip((k, v), after[i]):
                    np.testing.assert_array_equal(f(y[r])[:kept], tree.commit(x, before[r], path[r].tolist(), int(n[r]))[:kept])
            assert int(grown[r]) == before[r] + int(n[r]) + 1
        length.copy_(grown)
