"""The operators of one verification step of a drafted tree over a paged key/value cache, as cases to measure.

Each case is one call of one operator: the tree's mask and positions, the rotary positions with the
append to the cache, the attention of the drafted nodes, the walk along the target's choices, and the
commit of the accepted nodes' cache rows. `run` computes it in elementary torch operations in 32
bits, or, with `own`, by the library's call.
"""
import math

import numpy as np
import torch

own = False

GOLD = 0.6180339887498949


def listed():
    return [
        # a few requests with small trees, as in an interactive service: latency
        {"name": "mask_small", "op": "mask", "R": 4, "T": 16},
        # a full batch of wide trees
        {"name": "mask_wide", "op": "mask", "R": 256, "T": 512},
        # one decoding step of eight chats: one token each, text positions on one axis
        {"name": "rope_token", "op": "rope", "R": 8, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "axes": 1,
         "inter": False, "page": 16, "lo": 100, "hi": 900, "bf16": True},
        # the prefill of two documents with page images: positions on three axes, odd length
        {"name": "rope_image", "op": "rope", "R": 2, "T": 6001, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "axes": 3,
         "inter": False, "page": 64, "lo": 0, "hi": 40, "bf16": True},
        # one user, one token, a few thousand tokens of context: latency
        {"name": "att_token", "op": "att", "R": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "lo": 4097, "hi": 4097,
         "softcap": 0.0, "chain": True, "bf16": True},
        # 32 requests verifying blocks of seven drafted tokens after the last verified one, ragged contexts
        {"name": "att_block", "op": "att", "R": 32, "T": 8, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "lo": 300, "hi": 8200,
         "softcap": 0.0, "chain": True, "bf16": True},
        # long contexts with trees of 64 nodes, eight query heads per key head and capped scores
        {"name": "att_tree", "op": "att", "R": 4, "T": 64, "Hq": 32, "Hkv": 4, "D": 128, "page": 128, "lo": 40000, "hi": 65600,
         "softcap": 50.0, "chain": False, "bf16": True},
        # a 32-bit model on odd sizes: three query heads per key head, 80 columns, pages of 24
        {"name": "att_f32", "op": "att", "R": 6, "T": 13, "Hq": 12, "Hkv": 4, "D": 80, "page": 24, "lo": 0, "hi": 1500,
         "softcap": 30.0, "chain": False, "bf16": False},
        # a few requests with small trees: latency
        {"name": "accept_small", "op": "accept", "R": 8, "T": 16},
        # a full batch of wide trees
        {"name": "accept_wide", "op": "accept", "R": 512, "T": 512},
        # one request's branch moved in two layers: latency
        {"name": "commit_small", "op": "commit", "R": 1, "T": 16, "L": 2, "Hkv": 8, "D": 128, "page": 16, "lo": 500, "hi": 500, "bf16": True},
        # 64 requests' accepted branches moved in 16 layers at once
        {"name": "commit_batch", "op": "commit", "R": 64, "T": 64, "L": 16, "Hkv": 8, "D": 128, "page": 64, "lo": 33, "hi": 300, "bf16": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(["mask", "rope", "att", "att", "att", "accept", "commit"])
    if op in ("mask", "accept"):
        return {"op": op, "R": _log(rng, 1, 512 if op == "accept" else 256), "T": _log(rng, 2, 512)}
    bf16 = rng.random() < 0.75
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 80, 96, 128])
    page = rng.choice([16, 24, 32, 64, 128])
    if op == "rope":
        R = _log(rng, 1, 64)
        return {"op": op, "R": R, "T": _log(rng, 1, 12000 // R), "Hq": Hkv * rng.choice([1, 2, 3, 4]), "Hkv": Hkv, "D": D,
                "rot": rng.choice([D, D // 2]), "axes": rng.choice([1, 3]), "inter": rng.random() < 0.5, "page": page, "lo": 0,
                "hi": _log(rng, 1, 2000), "bf16": bf16}
    if op == "commit":
        return {"op": op, "R": _log(rng, 1, 64), "T": _log(rng, 2, 64), "L": _log(rng, 1, 16), "Hkv": Hkv, "D": D, "page": page,
                "lo": 0, "hi": _log(rng, 1, 300), "bf16": bf16}
    G = rng.choice([1, 2, 3, 4, 5, 8])
    R, T = _log(rng, 1, 64), _log(rng, 1, 100)
    if bf16:                                             # scores of the plain form and keys stay below the largest listed case's
        most = min((4 * 32 * 64 * 50000) // (R * Hkv * G * T), (4 * 4 * 128 * 50000) // (R * Hkv * D), 65600)
    else:
        most = min((64 * 78 * 12 * 1500) // (R * Hkv * G * T), 8000)
    hi = _log(rng, 1, max(1, most))
    return {"op": "att", "R": R, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "lo": hi // 4, "hi": hi,
            "softcap": rng.choice([0.0, 0.0, 30.0]), "chain": rng.random() < 0.4, "bf16": bf16}


def _lens(case):
    """Ragged committed lengths, the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo) * ((r + 1) * GOLD % 1.0) + 0.5) for r in range(case["R"])]


def _nodes(case):
    """Ragged node counts: every other request has fewer than T."""
    T = case["T"]
    return [T if r % 2 == 0 else T - int((T - 1) * (r * GOLD % 1.0) / 2) for r in range(case["R"])]


def _accepted(case):
    """Accepted drafted nodes of the commit's requests."""
    T = case["T"]
    return [min(T // 4, 1 + int(12 * ((r + 1) * GOLD % 1.0))) for r in range(case["R"])]


def work(case):
    op, R, T = case["op"], case["R"], case["T"]
    words = (T + 31) // 32
    if op == "mask":
        return {"bytes": 4 * R * T * (2 + words) + 8 * R, "flops": 0}
    if op == "accept":
        return {"bytes": 4 * R * T * 5 + 8 * R, "flops": 0}
    e = 2 if case["bf16"] else 4
    D, Hkv = case["D"], case["Hkv"]
    if op == "commit":
        rows = sum(_accepted(case))
        return {"bytes": rows * case["L"] * Hkv * D * e * 4, "flops": 0}
    n, c = _nodes(case), _lens(case)
    if op == "rope":
        rows = sum(n)
        per = (2 * case["Hq"] + 4 * Hkv) * D * e + 4 * case["rot"] + 4 * case["axes"]
        return {"bytes": rows * per, "flops": rows * (case["Hq"] + Hkv) * case["rot"] * 3}
    Hq = case["Hq"]
    keys = sum(a + b for a, b in zip(n, c))
    return {"bytes": keys * Hkv * D * e * 2 + sum(n) * Hq * (2 * D * e + 4) + 4 * R * T * words,
            "flops": 4 * D * Hq * sum(a * (b + 1) for a, b in zip(n, c))}


def _parents(case, gen):
    """Random trees: node 0 is the root, a node's parent is one of the few nodes before it."""
    R, T = case["R"], case["T"]
    i = torch.arange(T)
    back = 1 + (torch.rand((R, T), generator=gen) ** 2 * 6).long()
    p = (i - back).clamp(min=0)
    p[:, 0] = -1
    return p.int()


def _closure(parent, n):
    """[R, T, T] truth values: node j is node i or an ancestor of it; rows past the node count are empty."""
    R, T = parent.shape
    i = torch.arange(T, device=parent.device)
    live = i[None, :] < n[:, None].long()
    # slot T is the parent of the roots, and its own
    up = torch.where(parent < 0, T, parent.long())
    up = torch.cat([up, torch.full((R, 1), T, device=parent.device)], 1)
    anc = torch.eye(T + 1, T, dtype=torch.bool, device=parent.device).expand(R, T + 1, T)
    for _ in range(max(1, (T - 1).bit_length())):            # pointer doubling
        anc = anc | torch.gather(anc, 1, up[:, :, None].expand(R, T + 1, T))
        up = torch.gather(up, 1, up)
    return anc[:, :T] & live[:, :, None]


def _words(bits):
    """Packs [..., T] truth values into int32 words, bit j of word w being entry 32 w + j."""
    T = bits.shape[-1]
    w = (T + 31) // 32
    b = torch.nn.functional.pad(bits, (0, 32 * w - T)).reshape(*bits.shape[:-1], w, 32).long()
    v = (b << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).int()


def _bits(words, T):
    b = (words.long()[..., None] >> torch.arange(32, device=words.device)) & 1
    return b.flatten(-2)[..., :T].bool()


def _cache(case, gen, extra, layers=0):
    """A page table in random order over a pool with a few pages to spare, and the pool's keys and values."""
    R, page = case["R"], case["page"]
    per = [-(-(c + extra) // page) for c in _lens(case)]
    most, total = max(per), sum(per)
    order = torch.randperm(total + 3, generator=gen)
    table = torch.zeros((R, most), dtype=torch.int32)
    at = 0
    for r, k in enumerate(per):
        table[r, :k] = order[at:at + k].int()
        at += k
    shape = (total + 3, page, case["Hkv"], case["D"])
    shape = (layers,) + shape if layers else shape
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 40, (1,), generator=gen)))
    k = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    v = torch.randn(shape, dtype=dt, device="cuda", generator=g)
    return table.cuda(), k, v, g


def prepare(case, seed):
    op, R, T = case["op"], case["R"], case["T"]
    gen = torch.Generator().manual_seed(1000003 * int(seed) + 17 * R + T)
    s = {"op": op, "case": case}
    if op == "mask":
        s["parent"] = _parents(case, gen).cuda()
        s["n"] = torch.tensor(_nodes(case), dtype=torch.int32).cuda()
        s["base"] = torch.randint(0, 60000, (R,), generator=gen).int().cuda()
        s["out"] = (torch.empty((R, T, (T + 31) // 32), dtype=torch.int32, device="cuda"), torch.empty((R, T), dtype=torch.int32, device="cuda"))
    elif op == "accept":
        # the target agrees with a drafted child at most nodes, so walks run several nodes deep
        parent = _parents(case, gen)
        tokens = torch.randint(0, 4, (R, T), generator=gen).int()
        best = torch.randint(0, 5, (R, T), generator=gen).int()
        s["parent"], s["tokens"], s["best"] = parent.cuda(), tokens.cuda(), best.cuda()
        s["n"] = torch.tensor(_nodes(case), dtype=torch.int32).cuda()
        s["out"] = tuple(torch.empty(z, dtype=torch.int32, device="cuda") for z in ((R, T), (R,), (R, T)))
    elif op == "commit":
        # a side branch is accepted: the root, then nodes past every slot that is written
        acc = _accepted(case)
        path = torch.full((R, T), -1, dtype=torch.int32)
        for r, a in enumerate(acc):
            path[r, 0] = 0
            path[r, 1:a + 1] = (a + 1 + torch.randperm(T - a - 1, generator=gen)[:a].sort().values).int()
        s["table"], s["k"], s["v"], _ = _cache(case, gen, T, case["L"])
        s["ctx"] = torch.tensor(_lens(case), dtype=torch.int32).cuda()
        s["path"], s["acc"] = path.cuda(), torch.tensor(acc, dtype=torch.int32).cuda()
        s["new_len"] = torch.empty((R,), dtype=torch.int32, device="cuda")
    else:
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        dt = torch.bfloat16 if case["bf16"] else torch.float32
        s["table"], s["k"], s["v"], g = _cache(case, gen, T)
        s["ctx"] = torch.tensor(_lens(case), dtype=torch.int32).cuda()
        s["n"] = torch.tensor(_nodes(case), dtype=torch.int32).cuda()
        qkv = torch.randn((R, T, Hq + 2 * Hkv, D), dtype=dt, device="cuda", generator=g)   # one projection's rows
        s["q"], s["nk"], s["nv"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        if op == "rope":
            rot, A = case["rot"], case["axes"]
            far = 16384
            f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
            ang = torch.arange(far, dtype=torch.float64)[:, None] * f
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
            s["pos"] = torch.randint(0, far, (R, T, A), generator=gen).int().cuda()
            s["axis"] = (torch.arange(rot // 2) * A // (rot // 2)).int().cuda()
        else:
            parent = torch.arange(-1, T - 1).int().expand(R, T) if case["chain"] else _parents(case, gen)
            s["mask"] = _words(_closure(parent.cuda(), s["n"]))
            s["scale"] = 1.5 / math.sqrt(D)
        s["out"] = torch.empty((R, T, Hq, D), dtype=dt, device="cuda")
        s["lse"] = torch.empty((R, T, Hq), dtype=torch.float32, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own and op == "att":                                  # the workspace that a serving loop keeps
        import dspark_draft_selection_gb300 as ds
        s["ws"] = ds.workspace(ds.OP_TREE_ATTENTION, R, T, Hq * D, Hkv)
    return s


def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _own_mask(s):
    import dspark_draft_selection_gb300 as ds
    return ds.dspark_tree_mask(s["parent"], n_nodes=s["n"], base=s["base"], out=s["out"], status=s["status"])[:2]


def _own_rope(s):
    import dspark_draft_selection_gb300 as ds
    ds.dspark_rope_append(s["q"], s["nk"], s["nv"], s["pos"], s["cos_sin"], s["k"], s["v"], s["table"], s["ctx"], axis=s["axis"],
                          n_nodes=s["n"], interleaved=s["case"]["inter"], out=s["out"], status=s["status"])
    return s["out"], s["k"], s["v"]


def _own_att(s):
    import dspark_draft_selection_gb300 as ds
    return ds.dspark_tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], mask=s["mask"], n_nodes=s["n"], scale=s["scale"],
                                    softcap=s["case"]["softcap"], out=s["out"], lse=s["lse"], ws=s["ws"], status=s["status"])[:2]


def _own_accept(s):
    import dspark_draft_selection_gb300 as ds
    return ds.dspark_tree_accept(s["tokens"], s["parent"], s["best"], n_nodes=s["n"], out=s["out"], status=s["status"])[:3]


def _own_commit(s):
    import dspark_draft_selection_gb300 as ds
    ds.dspark_cache_commit(s["k"], s["v"], s["table"], s["ctx"], s["path"], s["acc"], out=s["new_len"], status=s["status"])
    return s["new_len"], s["k"], s["v"]


def _plain_mask(s):
    a = _closure(s["parent"], s["n"])
    depth = a.sum(-1) - 1
    return _words(a), torch.where(depth >= 0, s["base"][:, None] + depth, 0).int()


def _slots(s, i):
    """Page and place in the page of cache slot ctx + i of every request; i is [R, n]."""
    page = s["case"]["page"]
    at = s["ctx"][:, None].long() + i
    most = s["table"].shape[1] - 1
    return torch.gather(s["table"].long(), 1, (at // page).clamp(max=most)), at % page


def _rotate(x, c, sn, rot, inter):
    x = x.float()
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    c, sn = c[:, :, None], sn[:, :, None]
    y[..., a] = x[..., a] * c - x[..., b] * sn
    y[..., b] = x[..., b] * c + x[..., a] * sn
    return y


def _plain_rope(s):
    case = s["case"]
    rot, h = case["rot"], case["rot"] // 2
    at = s["pos"].long()[:, :, s["axis"].long()]
    f = torch.arange(h, device="cuda")
    c, sn = s["cos_sin"][at, f], s["cos_sin"][at, h + f]
    i = torch.arange(case["T"], device="cuda").expand(case["R"], -1)
    live = i < s["n"][:, None]
    q = _rotate(s["q"], c, sn, rot, case["inter"]).to(s["q"].dtype)
    k = _rotate(s["nk"], c, sn, rot, case["inter"]).to(s["q"].dtype)
    p, o = _slots(s, i)
    s["k"][p[live], o[live]] = k[live]
    s["v"][p[live], o[live]] = s["nv"][live]
    return torch.where(live[:, :, None, None], q, 0), s["k"], s["v"]


def _gather(s, cache, at):
    page = s["case"]["page"]
    p = torch.gather(s["table"].long(), 1, (at // page).clamp(max=s["table"].shape[1] - 1))
    return cache[p, at % page]


def _plain_att(s):
    case = s["case"]
    R, T, Hkv, D = case["R"], case["T"], case["Hkv"], case["D"]
    G = case["Hq"] // Hkv
    S = max(_lens(case)) + T
    j = torch.arange(S, device="cuda").expand(R, S)
    end = s["ctx"] + s["n"]
    k = _gather(s, s["k"], j).float().permute(0, 2, 3, 1)                       # [R, Hkv, D, S]
    q = s["q"].float().reshape(R, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * T, D)
    x = torch.matmul(q, k) * s["scale"]
    del k
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    node = (j - s["ctx"][:, None]).long()                                       # [R, S]
    seen = torch.gather(_bits(s["mask"], T), 2, node.clamp(0, T - 1)[:, None, :].expand(R, T, S))
    i = torch.arange(T, device="cuda")
    seen = ((node < 0)[:, None] | (seen & (j < end[:, None])[:, None])) & (i[None, :] < s["n"][:, None])[:, :, None]
    seen = seen[:, None, None].expand(R, Hkv, G, T, S)
    x = torch.where(seen, x.reshape(R, Hkv, G, T, S), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    v = _gather(s, s["v"], j).float().permute(0, 2, 1, 3)                       # [R, Hkv, S, D]
    o = torch.matmul(x.reshape(R, Hkv, G * T, S), v).reshape(R, Hkv, G, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(R, T, Hkv * G, D).to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(R, T, Hkv * G)


def _plain_accept(s):
    R, T = s["parent"].shape
    i = torch.arange(T, device="cuda")
    live = i < s["n"][:, None]
    p = s["parent"].long()
    hit = (s["tokens"] == torch.gather(s["best"], 1, p.clamp(min=0))) & (p >= 0) & live
    # of the children that match, the lowest index is followed
    rank = torch.full((R, T), T, device="cuda").scatter_reduce(1, p.clamp(min=0), torch.where(hit, i, T), "amin")
    hit = hit & (torch.gather(rank, 1, p.clamp(min=0)) == i)
    hit[:, 0] = live[:, 0]
    anc = _closure(s["parent"], s["n"])
    on = live & ~(anc & ~hit[:, None, :]).any(-1) & anc[:, :, 0]
    path = torch.where(on, i, T).sort(-1).values
    acc = on.sum(-1) - 1
    there = path < T
    tokens = torch.gather(s["tokens"], 1, path.clamp(max=T - 1))
    last = torch.gather(path, 1, acc.clamp(min=0)[:, None])
    best = torch.gather(s["best"], 1, last.clamp(max=T - 1))
    out = torch.where(there[:, 1:], tokens[:, 1:], -1)
    out = torch.cat([out, torch.full((R, 1), -1, device="cuda", dtype=torch.int32)], 1)
    out = torch.where(i == acc[:, None], best, out)
    return out, acc.int(), torch.where(there, path, -1).int()


def _plain_commit(s):
    R, T = s["path"].shape
    i = torch.arange(T, device="cuda").expand(R, T)
    move = i <= s["acc"][:, None]
    ps, os_ = _slots(s, s["path"].long().clamp(min=0))
    pd, od = _slots(s, i)
    ps, os_, pd, od = ps[move], os_[move], pd[move], od[move]
    s["k"][:, pd, od] = s["k"][:, ps, os_]
    s["v"][:, pd, od] = s["v"][:, ps, os_]
    return s["ctx"] + s["acc"] + 1, s["k"], s["v"]


_run_plain = {"mask": _plain_mask, "rope": _plain_rope, "att": _plain_att, "accept": _plain_accept, "commit": _plain_commit}
_run_own = {"mask": _own_mask, "rope": _own_rope, "att": _own_att, "accept": _own_accept, "commit": _own_commit}


def exact(case, seed):
    """The same outputs from the definitions, node by node or request by request, in 64 bits."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op, R, T = case["op"], case["R"], case["T"]
    if op == "mask":
        parent, n, base = (s[k].cpu().numpy() for k in ("parent", "n", "base"))
        mask, pos = np.zeros((R, T, (T + 31) // 32), np.uint32), np.zeros((R, T), np.int32)
        for r in range(R):
            for i in range(n[r]):
                p = parent[r, i]
                if p >= 0:
                    mask[r, i], pos[r, i] = mask[r, p], pos[r, p] + 1
                else:
                    pos[r, i] = base[r]
                mask[r, i, i // 32] |= np.uint32(1 << (i % 32))
        return mask.view(np.int32), pos
    if op == "accept":
        parent, tokens, best, n = (s[k].cpu().numpy() for k in ("parent", "tokens", "best", "n"))
        out, acc, path = np.full((R, T), -1, np.int32), np.zeros(R, np.int32), np.full((R, T), -1, np.int32)
        for r in range(R):
            cur, k, path[r, 0] = 0, 0, 0
            for i in range(1, n[r]):                         # a child comes after its parent
                if parent[r, i] == cur and tokens[r, i] == best[r, cur]:
                    out[r, k], cur = tokens[r, i], i
                    k += 1
                    path[r, k] = i
            out[r, k], acc[r] = best[r, cur], k
        return out, acc, path
    ctx, table, page = s["ctx"].tolist(), s["table"].cpu().numpy(), case["page"]
    where = lambda r, at: (int(table[r, at // page]), at % page)  # noqa: E731
    if op == "commit":
        path, acc = s["path"].tolist(), s["acc"].tolist()
        k, v = s["k"].clone(), s["v"].clone()
        for r in range(R):
            for i in range(acc[r] + 1):
                d, o = where(r, ctx[r] + i), where(r, ctx[r] + path[r][i])
                k[:, d[0], d[1]], v[:, d[0], d[1]] = s["k"][:, o[0], o[1]], s["v"][:, o[0], o[1]]
        return np.array([c + a + 1 for c, a in zip(ctx, acc)], np.int32), k, v
    n = s["n"].tolist()
    if op == "rope":
        h = case["rot"] // 2
        tab = s["cos_sin"].double()
        turn = torch.complex(tab[:, :h], tab[:, h:])
        axis = s["axis"].long()

        def spin(x, w):
            x = x.double()
            if case["inter"]:
                z = torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:-1], h, 2).contiguous()) * w
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * w
                y = torch.cat([z.real, z.imag], -1)
            return torch.cat([y, x[..., 2 * h:]], -1)

        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        k, v = s["k"].double(), s["v"].double()
        for r in range(R):
            p = s["pos"][r, :n[r]].long()[:, axis]
            w = turn[p, torch.arange(h, device="cuda")][:, None]
            q[r, :n[r]] = spin(s["q"][r, :n[r]], w)
            at = torch.arange(ctx[r], ctx[r] + n[r], device="cuda")
            where_r = s["table"][r].long()[at // page], at % page
            k[where_r], v[where_r] = spin(s["nk"][r, :n[r]], w), s["nv"][r, :n[r]].double()
        return q, k, v
    Hkv, Hq, D = case["Hkv"], case["Hq"], case["D"]
    G = Hq // Hkv
    if sum(a * b for a, b in zip(ctx, n)) * Hq * D > 6e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for r in range(R):
        at = torch.arange(ctx[r] + n[r], device="cuda")
        pg = s["table"][r].long()[at // page], at % page
        kr, vr = s["k"][pg].double(), s["v"][pg].double()
        ok = torch.ones((n[r], ctx[r] + n[r]), dtype=torch.bool, device="cuda")
        ok[:, ctx[r]:] = _bits(s["mask"][r, :n[r]], T)[:, :n[r]]
        for hd in range(Hq):
            x = s["q"][r, :n[r], hd].double() @ kr[:, hd // G].T * s["scale"]
            x = case["softcap"] * torch.tanh(x / case["softcap"]) if case["softcap"] else x
            x = x.masked_fill(~ok, -math.inf)
            lse[r, :n[r], hd] = torch.logsumexp(x, -1)
            out[r, :n[r], hd] = torch.nan_to_num(torch.softmax(x, -1)) @ vr[:, hd // G]
    return out, lse
