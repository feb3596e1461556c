"""Speculative decoding with drafted trees over a paged cache, on a small random float32 transformer.

Each step drafts a tree (a chain of the best candidates of every position with the second best as leaves,
from dspark_topk), runs the target on all its nodes at once (dspark_tree_mask, then in every layer
dspark_rope_append and dspark_tree_attention), takes the target's choices (dspark_topk with K = 1), walks
them (dspark_tree_accept) and keeps the accepted rows of the cache (dspark_cache_commit). The tokens are
those of decoding one token at a time; `python examples/tree_step.py` checks that and prints how many
target passes the trees saved.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dspark_draft_selection_gb300 as ds  # noqa: E402


class Target:
    """A random decoder: layers of attention over the paged cache and a gated product, all float32."""

    def __init__(self, R, vocab=500, layers=3, Hq=8, H=2, D=64, page=16, tokens=256, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        w = lambda *s: torch.randn(s, device="cuda", generator=g) * s[0] ** -0.5  # noqa: E731
        self.R, self.Hq, self.H, self.D, self.layers, d = R, Hq, H, D, layers, Hq * D
        self.embed, self.head = w(vocab, d) * vocab ** 0.5, w(d, vocab)
        self.qkv = [w(d, (Hq + 2 * H) * D) for _ in range(layers)]
        self.o, self.up, self.down = ([w(*s) for _ in range(layers)] for s in ((d, d), (d, 2 * d), (2 * d, d)))
        per = tokens // page
        shape = (layers, R * per, page, H, D)
        self.k, self.v = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
        order = torch.randperm(R * per, generator=torch.Generator().manual_seed(seed))
        self.table = order.int().reshape(R, per).cuda()
        f = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
        a = torch.arange(tokens, dtype=torch.float64)[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.length = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.status = ds.new_status()

    def __call__(self, tokens, parent=None):
        """The target's choice after each node of the trees (tokens, parent [R, T]; None: chains); the nodes'
        keys and values are then in the cache behind the committed tokens."""
        R, T = tokens.shape
        mask, pos, _ = ds.dspark_tree_mask(parent, R=R, T=T, base=self.length, status=self.status)
        x = self.embed[tokens.long()]
        ws = ds.workspace(ds.OP_TREE_ATTENTION, R, T, self.Hq * self.D, self.H)
        for i in range(self.layers):
            y = torch.nn.functional.layer_norm(x, x.shape[-1:]) @ self.qkv[i]
            q, k, v = y.reshape(R, T, -1, self.D).split([self.Hq, self.H, self.H], 2)
            q, _ = ds.dspark_rope_append(q, k, v, pos, self.cos_sin, self.k[i], self.v[i], self.table, self.length,
                                         status=self.status)
            a, _, _ = ds.dspark_tree_attention(q, self.k[i], self.v[i], self.table, self.length, mask=mask, lse=False, ws=ws,
                                               status=self.status)
            x = x + a.reshape(R, T, -1) @ self.o[i]
            x = x + torch.relu(torch.nn.functional.layer_norm(x, x.shape[-1:]) @ self.up[i]) @ self.down[i]
        logits = torch.nn.functional.layer_norm(x, x.shape[-1:]) @ self.head
        return ds.dspark_topk(logits.reshape(R * T, -1), T, 1, status=self.status)[1].reshape(R, T)

    def keep(self, path, n_accepted):
        """Keeps the accepted nodes in every layer."""
        self.length, _ = ds.dspark_cache_commit(self.k, self.v, self.table, self.length, path, n_accepted, T=1, status=self.status)


def one_by_one(R, prompt, steps, **kw):
    """Greedy decoding, one token a pass: [R, steps]."""
    t = Target(R, **kw)
    zero = torch.zeros(R, dtype=torch.int32, device="cuda")
    last = prompt[:, 0].contiguous()
    out = []
    for _ in range(steps):
        last = t(last[:, None].contiguous())[:, 0].contiguous()
        t.keep(None, zero)
        out.append(last)
    assert ds.read_status(t.status) == 0
    return torch.stack(out, 1)


def with_trees(R, prompt, want, block=5, hit=0.7, seed=1, **kw):
    """The same tokens by drafted trees; the draft's logits are noise with the right token raised at a share
    `hit` of the places, and second at most others. Returns (tokens [R, steps], target passes)."""
    t = Target(R, **kw)
    steps, vocab = want.shape[1], t.head.shape[1]
    g = torch.Generator("cuda").manual_seed(seed)
    out = [[] for _ in range(R)]
    last = prompt[:, 0].contiguous()
    passes = 0
    # node 0 is the last token, nodes 1..block the best candidates, block + j the second best of position j
    parent = torch.tensor([-1] + list(range(block)) + list(range(block)), dtype=torch.int32, device="cuda").expand(R, -1).contiguous()
    while min(map(len, out)) < steps:
        logits = torch.randn((R, block, vocab), device="cuda", generator=g)
        at = torch.tensor([len(o) for o in out], device="cuda")[:, None] + torch.arange(block, device="cuda")
        right = want.gather(1, at.clamp(max=steps - 1)).long()[:, :, None]
        logits.scatter_(2, torch.randint(0, vocab, right.shape, device="cuda", generator=g), 8.0)
        logits.scatter_(2, right, torch.where(torch.rand(right.shape, device="cuda", generator=g) < hit, 9.0, 7.0))
        cand = ds.dspark_topk(logits.reshape(R * block, vocab), block, 2, status=t.status)[1]
        tokens = torch.cat([last[:, None], cand[:, :, 0], cand[:, :, 1]], 1).contiguous()
        best = t(tokens, parent)
        new, n, path, _ = ds.dspark_tree_accept(tokens, parent, best, status=t.status)
        t.keep(path, n)
        last = new.gather(1, n.long()[:, None])[:, 0].contiguous()
        for r, (row, k) in enumerate(zip(new.tolist(), n.tolist())):
            out[r] += row[:k + 1]
        passes += 1
    assert ds.read_status(t.status) == 0
    return torch.tensor([o[:steps] for o in out], dtype=torch.int32), passes


def main(R=4, steps=40):
    prompt = torch.arange(1, R + 1, dtype=torch.int32, device="cuda")[:, None]
    want = one_by_one(R, prompt, steps)
    got, passes = with_trees(R, prompt, want)
    assert torch.equal(got, want.cpu()), "the trees' tokens are not those of decoding one by one"
    print(f"{R} requests x {steps} tokens: the same tokens in {passes} target passes instead of {steps}")
    return steps, passes


if __name__ == "__main__":
    main()
