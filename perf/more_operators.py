"""The operators of a drafted tree's verification step over a key/value cache kept in 8 bits, as cases to measure.

Each case is one call of one operator: the rotary positions with the quantising append, the attention of
the drafted nodes (or of one new token) over the codes, the commit of the accepted nodes' rows, the read back
into 16 or 32 bits, and the sampled acceptance along the tree from given random numbers. `run` computes it in elementary
torch operations, or, with `own`, by the library's call.

The cache: blocks of 32 columns of a head share a power of two 2^e, e + 127 in one byte; a column's value is
its code (e4m3 or a whole number from -127 to 127) times 2^e.
"""
import math

import numpy as np
import torch

own = False

GOLD = 0.6180339887498949


def listed():
    return [
        # one decoding step of eight chats: one token each, text positions on one axis: latency
        {"name": "append_token", "op": "append", "R": 8, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "axes": 1, "inter": False,
         "page": 16, "lo": 100, "hi": 900, "bf16": True, "e4m3": True, "by_head": True},
        # the prefill of three documents with page images: positions on three axes, odd length
        {"name": "append_image", "op": "append", "R": 3, "T": 4999, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "axes": 3, "inter": False,
         "page": 64, "lo": 0, "hi": 40, "bf16": True, "e4m3": False, "by_head": True},
        # the first pages of one conversation handed to a 32-bit tool: latency
        {"name": "read_prefix", "op": "read", "R": 1, "Hkv": 8, "D": 128, "page": 16, "lo": 333, "hi": 333, "from": 0, "bf16": False,
         "e4m3": True, "by_head": True},
        # a batch of ragged conversations read back from a shared prefix on, for attention in 16 bits
        {"name": "read_batch", "op": "read", "R": 32, "Hkv": 8, "D": 128, "page": 64, "lo": 300, "hi": 8200, "from": 37, "bf16": True,
         "e4m3": False, "by_head": True},
        # one user, one token, a few thousand tokens of context: latency
        {"name": "att_token", "op": "att", "R": 1, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "lo": 5001, "hi": 5001,
         "softcap": 0.0, "chain": True, "bf16": True, "e4m3": True, "by_head": True},
        # a full batch of single new tokens over ragged contexts
        {"name": "att_batch", "op": "att", "R": 64, "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "lo": 300, "hi": 8200,
         "softcap": 0.0, "chain": True, "bf16": True, "e4m3": False, "by_head": True},
        # 32 requests verifying blocks of seven drafted tokens after the last verified one, ragged contexts
        {"name": "att_block", "op": "att", "R": 32, "T": 8, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "lo": 300, "hi": 8200,
         "softcap": 0.0, "chain": True, "bf16": True, "e4m3": True, "by_head": True},
        # long contexts with trees of 64 nodes, eight query heads per key head and capped scores
        {"name": "att_tree", "op": "att", "R": 4, "T": 64, "Hq": 32, "Hkv": 4, "D": 128, "page": 128, "lo": 40000, "hi": 65600,
         "softcap": 50.0, "chain": False, "bf16": True, "e4m3": True, "by_head": True},
        # one request's branch moved in two layers: latency
        {"name": "commit_small", "op": "commit", "R": 1, "T": 16, "L": 2, "Hkv": 8, "D": 128, "page": 16, "lo": 500, "hi": 500, "e4m3": True,
         "by_head": True},
        # 64 requests' accepted branches moved in 16 layers at once
        {"name": "commit_batch", "op": "commit", "R": 64, "T": 64, "L": 16, "Hkv": 8, "D": 128, "page": 64, "lo": 33, "hi": 300, "e4m3": False,
         "by_head": True},
        # one user's tree of the best candidates, no proposal distribution: latency
        {"name": "verify_best", "op": "verify", "R": 1, "T": 16, "V": 151936, "proposal": False},
        # a batch of trees drawn from their proposals
        {"name": "verify_drawn", "op": "verify", "R": 64, "T": 24, "V": 151936, "proposal": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(["append", "read", "att", "att", "att", "commit", "verify"])
    if op == "verify":
        V = _log(rng, 500, 151936)
        R = _log(rng, 1, 64)
        return {"op": op, "R": R, "T": _log(rng, 2, max(2, min(64, 64 * 24 * 151936 // (R * V)))), "V": V, "proposal": rng.random() < 0.5}
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 80, 96, 128])
    base = {"op": op, "Hkv": Hkv, "D": D, "page": rng.choice([16, 24, 32, 64, 128]), "e4m3": rng.random() < 0.5, "by_head": rng.random() < 0.7}
    bf16 = rng.random() < 0.75
    if op == "append":
        R = _log(rng, 1, 64)
        return dict(base, R=R, T=_log(rng, 1, 12000 // R), Hq=Hkv * rng.choice([1, 2, 3, 4]), rot=rng.choice([D, D // 2]), axes=rng.choice([1, 3]),
                    inter=rng.random() < 0.5, lo=0, hi=_log(rng, 1, 2000), bf16=bf16)
    if op == "read":
        R = _log(rng, 1, 64)
        hi = _log(rng, 1, 100000 // R)
        return dict(base, R=R, lo=hi // 4, hi=hi, bf16=bf16, **{"from": rng.choice([0, 0, min(hi // 4, 100)])})
    if op == "commit":
        return dict(base, R=_log(rng, 1, 64), T=_log(rng, 4, 64), L=_log(rng, 1, 16), lo=0, hi=_log(rng, 1, 300))
    G = rng.choice([1, 2, 3, 4, 5, 8])
    R, T = _log(rng, 1, 64), rng.choice([1, _log(rng, 1, 100)])
    if bf16:                                             # scores of the plain form and keys stay below the largest listed case's
        most = min((4 * 32 * 64 * 50000) // (R * Hkv * G * T), (4 * 4 * 128 * 50000) // (R * Hkv * D), 65600)
    else:
        most = min((64 * 78 * 12 * 1500) // (R * Hkv * G * T), 8000)
    hi = _log(rng, 1, max(1, most))
    return dict(base, R=R, T=T, Hq=Hkv * G, lo=hi // 4, hi=hi, softcap=rng.choice([0.0, 0.0, 30.0]), chain=rng.random() < 0.4, bf16=bf16)


def _lens(case):
    """Ragged lengths, the same for every seed."""
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
    op, R = case["op"], case["R"]
    if op == "verify":                                   # the row that the last token is drawn from, and what names the nodes
        return {"bytes": R * case["V"] * 4 * (2 if case["proposal"] else 1) + R * case["T"] * (2 * 4 + 8 + 2 * 4), "flops": 0}
    D, Hkv = case["D"], case["Hkv"]
    row = 2 * Hkv * (D + -(-D // 32))                    # a slot's keys and values with their scales
    if op == "commit":
        return {"bytes": sum(_accepted(case)) * case["L"] * row * 2, "flops": 0}
    e = 2 if case["bf16"] else 4
    if op == "read":
        rows = sum(n - case["from"] for n in _lens(case))
        return {"bytes": rows * (row + 2 * Hkv * D * e), "flops": 0}
    Hq, T = case["Hq"], case["T"]
    n, c = _nodes(case), _lens(case)
    if op == "append":
        rows = sum(n)
        per = (2 * Hq + 2 * Hkv) * D * e + row + 4 * case["rot"] + 4 * case["axes"]
        return {"bytes": rows * per, "flops": rows * (Hq + Hkv) * case["rot"] * 3}
    keys = sum(a + b for a, b in zip(n, c))
    return {"bytes": keys * row + sum(n) * Hq * (2 * D * e + 4) + 4 * R * T * ((T + 31) // 32),
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


def _quantise(y, e4m3):
    """float32 y [..., D] -> (codes [..., D], scale bytes [..., blocks])."""
    D = y.shape[-1]
    nb = -(-D // 32)
    b = torch.nn.functional.pad(y, (0, 32 * nb - D)).unflatten(-1, (nb, 32))
    most = b.abs().amax(-1)
    f, k = torch.frexp(most)                             # f 2^k, f in [1/2, 1)
    # 448 = 0.875 * 2^9, 127 = 0.9921875 * 2^7
    e = torch.where(f <= 0.875, k - 9, k - 8) if e4m3 else torch.where(f <= 0.9921875, k - 7, k - 6)
    e = torch.where(most > 0, e, -126).clamp(-126, 118)
    z = b * ((127 - e) << 23).int().view(torch.float32)[..., None]
    z = z.flatten(-2)[..., :D]
    codes = z.clamp(-448, 448).to(torch.float8_e4m3fn) if e4m3 else z.round().clamp(-127, 127).to(torch.int8)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, scale):
    """The numbers in 32 bits that codes [..., D] under scale bytes [..., blocks] stand for (bytes 1..245)."""
    f = (scale.int() << 23).view(torch.float32)
    return codes.float() * f.repeat_interleave(32, -1)[..., :codes.shape[-1]]


def _cache(case, gen, extra, layers=0):
    """A page table in random order over a pool with a few pages to spare, and the pool's codes and scales."""
    R, page, Hkv, D = case["R"], case["page"], case["Hkv"], case["D"]
    per = [max(1, -(-(c + extra) // page)) for c in _lens(case)]
    most, total = max(per), sum(per)
    order = torch.randperm(total + 3, generator=gen)
    table = torch.zeros((R, most), dtype=torch.int32)
    at = 0
    for r, k in enumerate(per):
        table[r, :k] = order[at:at + k].int()
        at += k
    g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 40, (1,), generator=gen)))
    lead = (layers,) if layers else ()
    made = []
    for _ in range(2):
        c, s = _quantise(torch.randn(lead + (total + 3, page, Hkv, D), device="cuda", generator=g), case["e4m3"])
        if case["by_head"]:                              # the scales of a head's slots side by side
            s = s.transpose(-3, -2).contiguous().transpose(-3, -2)
        made.append((c, s))
    (k, ks), (v, vs) = made
    return table.cuda(), (k, v, ks, vs), g


def prepare(case, seed):
    op, R = case["op"], case["R"]
    gen = torch.Generator().manual_seed(1000003 * int(seed) + 17 * R + case.get("T", 0))
    s = {"op": op, "case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "verify":
        T, V = case["T"], case["V"]
        g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 40, (1,), generator=gen)))
        parent = _parents(case, gen).cuda()
        z = 2.0 * torch.randn((R, T, V), device="cuda", generator=g)
        t = z + 0.7 * torch.randn((R, T, V), device="cuda", generator=g)
        s["p"] = torch.softmax(t, -1)
        del t
        sib = torch.tril(parent[:, :, None] == parent[:, None, :], -1).sum(-1)        # earlier children of the same parent
        up, k = parent.long().clamp(min=0), min(8, V)
        if case["proposal"]:
            s["q"] = torch.softmax(z, -1)
            made = torch.multinomial(s["q"].reshape(R * T, V), k, replacement=True, generator=g).reshape(R, T, k)
        else:
            s["q"], made = None, z.topk(k, -1).indices
        del z
        s["parent"] = parent
        s["tokens"] = made[torch.arange(R, device="cuda")[:, None], up, sib.clamp(max=k - 1)].int()
        s["n"] = torch.tensor(_nodes(case), dtype=torch.int32).cuda()
        s["ua"] = torch.rand((R, T), dtype=torch.float64, device="cuda", generator=g)
        s["ud"] = torch.rand((R,), dtype=torch.float64, device="cuda", generator=g)
        s["out"] = tuple(torch.empty(z, dtype=torch.int32, device="cuda") for z in ((R, T), (R,), (R, T)))
        return s
    Hkv, D = case["Hkv"], case["D"]
    lens = torch.tensor(_lens(case), dtype=torch.int32)
    if op == "commit":
        # a side branch is accepted: the root, then nodes past every slot that is written
        T, acc = case["T"], _accepted(case)
        path = torch.full((R, T), -1, dtype=torch.int32)
        for r, a in enumerate(acc):
            path[r, 0] = 0
            path[r, 1:a + 1] = (a + 1 + torch.randperm(T - a - 1, generator=gen)[:a].sort().values).int()
        s["table"], s["cache"], _ = _cache(case, gen, T, case["L"])
        s["ctx"], s["path"], s["acc"] = lens.cuda(), path.cuda(), torch.tensor(acc, dtype=torch.int32).cuda()
        s["new_len"] = torch.empty((R,), dtype=torch.int32, device="cuda")
        return s
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    if op == "read":
        s["table"], s["cache"], _ = _cache(case, gen, 0)
        s["start"] = torch.full((R,), case["from"], dtype=torch.int32, device="cuda")
        s["n"] = (lens - case["from"]).cuda()
        S = max(_lens(case)) - case["from"]
        s["out"] = tuple(torch.zeros((R, max(1, S), Hkv, D), dtype=dt, device="cuda") for _ in range(2))
        return s
    T, Hq = case["T"], case["Hq"]
    s["table"], s["cache"], g = _cache(case, gen, T)
    s["ctx"] = lens.cuda()
    s["n"] = torch.tensor(_nodes(case), dtype=torch.int32).cuda()
    qkv = torch.randn((R, T, Hq + 2 * Hkv, D), dtype=dt, device="cuda", generator=g)       # one projection's rows
    s["q"], s["nk"], s["nv"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    if op == "append":
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
        s["lse"] = torch.empty((R, T, Hq), dtype=torch.float32, device="cuda")
        if own:                                          # the workspace that a serving loop keeps
            import dspark_draft_selection_gb300 as ds
            s["ws"] = ds.workspace(ds.OP_TREE_ATTENTION_Q8, R, T, Hq * D, Hkv)
    s["out"] = torch.empty((R, T, Hq, D), dtype=dt, device="cuda")
    return s


def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _own_append(s):
    import dspark_draft_selection_gb300 as ds
    ds.dspark_rope_append_q8(s["q"], s["nk"], s["nv"], s["pos"], s["cos_sin"], s["cache"], s["table"], s["ctx"], axis=s["axis"],
                             n_nodes=s["n"], interleaved=s["case"]["inter"], out=s["out"], status=s["status"])
    return (s["out"],) + s["cache"]


def _own_read(s):
    import dspark_draft_selection_gb300 as ds
    return ds.dspark_cache_read_q8(s["cache"], s["table"], s["n"], start=s["start"], out=s["out"], status=s["status"])[:2]


def _own_att(s):
    import dspark_draft_selection_gb300 as ds
    return ds.dspark_tree_attention_q8(s["q"], s["cache"], s["table"], s["ctx"], mask=s["mask"], n_nodes=s["n"], scale=s["scale"],
                                       softcap=s["case"]["softcap"], out=s["out"], lse=s["lse"], ws=s["ws"], status=s["status"])[:2]


def _own_commit(s):
    import dspark_draft_selection_gb300 as ds
    ds.dspark_cache_commit_q8(s["cache"], s["table"], s["ctx"], s["path"], s["acc"], out=s["new_len"], status=s["status"])
    return (s["new_len"],) + s["cache"]


def _own_verify(s):
    import dspark_draft_selection_gb300 as ds
    return ds.dspark_tree_verify(s["p"], s["tokens"], s["parent"], s["ua"], s["ud"], q=s["q"], n_nodes=s["n"], out=s["out"],
                                 status=s["status"])[:3]


def _slots(s, at):
    """Page and place in the page of slots `at` [R, n] of every request."""
    page = s["case"]["page"]
    e = (at // page).clamp(max=s["table"].shape[1] - 1)
    return torch.gather(s["table"].long(), 1, e), at % page


def _rotate(x, c, sn, rot, inter):
    """Every product and every sum rounded to 32 bits: what is quantised next depends on each."""
    x = x.float()
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    c, sn = c[:, :, None], sn[:, :, None]
    y[..., a] = x[..., a] * c - x[..., b] * sn
    y[..., b] = x[..., b] * c + x[..., a] * sn
    return y


def _plain_append(s):
    case = s["case"]
    rot, h = case["rot"], case["rot"] // 2
    at = s["pos"].long()[:, :, s["axis"].long()]
    f = torch.arange(h, device="cuda")
    c, sn = s["cos_sin"][at, f], s["cos_sin"][at, h + f]
    i = torch.arange(case["T"], device="cuda").expand(case["R"], -1)
    live = i < s["n"][:, None]
    q = _rotate(s["q"], c, sn, rot, case["inter"]).to(s["q"].dtype)
    k, ks = _quantise(_rotate(s["nk"], c, sn, rot, case["inter"])[live], case["e4m3"])
    v, vs = _quantise(s["nv"].float()[live], case["e4m3"])
    p, o = _slots(s, s["ctx"][:, None].long() + i)
    p, o = p[live], o[live]
    for cache, new in zip(s["cache"], (k, v, ks, vs)):
        cache.view(torch.uint8)[p, o] = new.view(torch.uint8)
    return (torch.where(live[:, :, None, None], q, 0),) + s["cache"]


def _gather(s, codes, scale, at):
    p, o = _slots(s, at)
    return _values(codes[p, o], scale[p, o])


def _plain_read(s):
    S = s["out"][0].shape[1]
    i = torch.arange(S, device="cuda").expand(s["case"]["R"], S)
    live = (i < s["n"][:, None])[:, :, None, None]
    k, v, ks, vs = s["cache"]
    at = s["start"][:, None].long() + i
    return tuple(torch.where(live, _gather(s, c, e, at), 0).to(o.dtype) for c, e, o in ((k, ks, s["out"][0]), (v, vs, s["out"][1])))


def _plain_att(s):
    case = s["case"]
    R, T, Hkv, D = case["R"], case["T"], case["Hkv"], case["D"]
    G = case["Hq"] // Hkv
    S = max(_lens(case)) + T
    j = torch.arange(S, device="cuda").expand(R, S)
    end = s["ctx"] + s["n"]
    kc, vc, ks, vs = s["cache"]
    k = _gather(s, kc, ks, j).permute(0, 2, 3, 1)                               # [R, Hkv, D, S]
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
    v = _gather(s, vc, vs, j).permute(0, 2, 1, 3)                               # [R, Hkv, S, D]
    o = torch.matmul(x.reshape(R, Hkv, G * T, S), v).reshape(R, Hkv, G, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(R, T, Hkv * G, D).to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(R, T, Hkv * G)


def _plain_commit(s):
    R, T = s["path"].shape
    i = torch.arange(T, device="cuda").expand(R, T)
    move = i <= s["acc"][:, None]
    ctx = s["ctx"][:, None].long()
    ps, os_ = _slots(s, ctx + s["path"].long().clamp(min=0))
    pd, od = _slots(s, ctx + i)
    ps, os_, pd, od = ps[move], os_[move], pd[move], od[move]
    for c in s["cache"]:
        c = c.view(torch.uint8)
        c[:, pd, od] = c[:, ps, os_]
    return (s["ctx"] + s["acc"] + 1,) + s["cache"]


def _plain_verify(s):
    """One look at each node in the order of their numbers, all requests at once: a node is tested where its parent is the
    node that the walk is on. Sums and tests in 64 bits, as a token is drawn where a sum passes a border."""
    p, q, tokens, parent = s["p"], s["q"], s["tokens"].long(), s["parent"]
    R, T, V = p.shape
    row = torch.arange(R, device="cuda")
    zero = torch.zeros(R, dtype=torch.long, device="cuda")
    cur, depth = zero, zero
    a, b = zero.double(), torch.ones(R, dtype=torch.float64, device="cuda")       # the residual is max(0, p - a q) / b
    left = p[row, cur].double()                                                   # unnormalised residual, 64 bits
    path = torch.full((R, T + 1), -1, device="cuda")
    path[:, 0] = 0
    out = torch.full((R, T + 1), -1, device="cuda")
    for i in range(1, T):
        x = tokens[:, i]
        asked = (parent[:, i] == cur) & (i < s["n"])
        qx = 1.0 if q is None else q[row, cur, x].double()
        yes = asked & (s["ua"][:, i] * b * qx < left[row, x])
        no = asked & ~yes
        if q is None:
            mass = b - left[row, x]
            left[row, x] = torch.where(no, 0.0, left[row, x])
        else:
            rest = (p[row, cur].double() - (a + b)[:, None] * q[row, cur].double()).clamp(min=0)
            left = torch.where(no[:, None], rest, left)
            mass = rest.sum(-1)
        a, b = torch.where(no, a + b, a), torch.where(no, mass, b)
        out[row, depth] = torch.where(yes, x, out[row, depth])
        depth = depth + yes
        path[row, depth] = torch.where(yes, i, path[row, depth])
        cur = torch.where(yes, i, cur)
        a, b = torch.where(yes, 0.0, a), torch.where(yes, 1.0, b)
        left = torch.where(yes[:, None], p[row, cur].double(), left)
    left = torch.where((left.sum(-1) > 0)[:, None], left, p[row, cur].double())
    run_ = left.cumsum(-1)
    past = (run_ > s["ud"][:, None] * run_[:, -1:]) & (left > 0)
    last = torch.where(left > 0, torch.arange(V, device="cuda"), -1).amax(-1)
    token = torch.where(past.any(-1), past.int().argmax(-1), last)
    out[row, depth] = token
    return out[:, :T].int(), depth.int(), path[:, :T].int()


_run_plain = {"append": _plain_append, "read": _plain_read, "att": _plain_att, "commit": _plain_commit, "verify": _plain_verify}
_run_own = {"append": _own_append, "read": _own_read, "att": _own_att, "commit": _own_commit, "verify": _own_verify}


def _number(codes, scale):
    """Values in 64 bits, block by block."""
    v = codes.double()
    two = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), scale.double() - 127)
    for b in range(scale.shape[-1]):
        v[..., 32 * b:32 * b + 32] *= two[..., b:b + 1]
    return v


def exact(case, seed):
    """The same outputs from the definitions, request by request, in 64 bits."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op, R = case["op"], case["R"]
    if op == "verify":                                   # whole numbers
        return None
    if op == "commit":
        return (None, _moved(s, 0), _moved(s, 1), None, None) if case["e4m3"] else None
    page, table = case["page"], s["table"].long()
    k, v, ks, vs = s["cache"]
    if op == "read":
        outs = tuple(torch.zeros(o.shape, dtype=torch.float64, device="cuda") for o in s["out"])
        for r, n in enumerate(s["n"].tolist()):
            at = torch.arange(case["from"], case["from"] + n, device="cuda")
            w = table[r, at // page], at % page
            outs[0][r, :n], outs[1][r, :n] = _number(k[w], ks[w]), _number(v[w], vs[w])
        return outs
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    ctx, n = s["ctx"].tolist(), s["n"].tolist()
    if op == "append":
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

        def codes(y):                                    # e4m3 numbers: three bits after the leading one, none below 2^-9
            out = torch.empty_like(y)
            for b in range(0, D, 32):
                z = y[..., b:b + 32]
                m = z.abs().amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(m / 448)).clamp(-126, 118)
                z = z * 2.0 ** -e
                step = 2.0 ** (torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
                out[..., b:b + 32] = torch.round(z / step) * step
            return out

        q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        kc, vc = (k.double(), v.double()) if case["e4m3"] else (None, None)
        for r in range(R):
            w = turn[s["pos"][r, :n[r]].long()[:, axis], torch.arange(h, device="cuda")][:, None]
            q[r, :n[r]] = spin(s["q"][r, :n[r]], w)
            if case["e4m3"]:
                at = torch.arange(ctx[r], ctx[r] + n[r], device="cuda")
                where = table[r, at // page], at % page
                kc[where], vc[where] = codes(spin(s["nk"][r, :n[r]], w)), codes(s["nv"][r, :n[r]].double())
        return q, kc, vc, None, None
    G = Hq // Hkv
    if sum(a * b for a, b in zip(ctx, n)) * Hq * D > 6e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for r in range(R):
        at = torch.arange(ctx[r] + n[r], device="cuda")
        pg = table[r, at // page], at % page
        kr, vr = _number(k[pg], ks[pg]), _number(v[pg], vs[pg])
        ok = torch.ones((n[r], ctx[r] + n[r]), dtype=torch.bool, device="cuda")
        ok[:, ctx[r]:] = _bits(s["mask"][r, :n[r]], T)[:, :n[r]]
        for hd in range(Hq):
            x = s["q"][r, :n[r], hd].double() @ kr[:, hd // G].T * s["scale"]
            x = case["softcap"] * torch.tanh(x / case["softcap"]) if case["softcap"] else x
            x = x.masked_fill(~ok, -math.inf)
            lse[r, :n[r], hd] = torch.logsumexp(x, -1)
            out[r, :n[r], hd] = torch.nan_to_num(torch.softmax(x, -1)) @ vr[:, hd // G]
    return out, lse


def _moved(s, which):
    """The codes of one buffer after the commit, row by row."""
    ctx, table, page = s["ctx"].tolist(), s["table"].cpu().numpy(), s["case"]["page"]
    old = s["cache"][which]
    new = old.double()
    src, dst = [], []
    for r, (path, a) in enumerate(zip(s["path"].tolist(), s["acc"].tolist())):
        for i in range(a + 1):
            f, t = ctx[r] + path[i], ctx[r] + i
            src.append((int(table[r, f // page]), f % page))
            dst.append((int(table[r, t // page]), t % page))
    (a, b), (c, d) = (tuple(torch.from_numpy(x).cuda() for x in np.array(w).T) for w in (src, dst))
    new[:, c, d] = old.double()[:, a, b]
    return new
