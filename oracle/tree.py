"""Trees of drafted nodes over a key/value cache (oracle; test infrastructure only): ancestor mask and
positions, rotary positions, attention, greedy acceptance and the commit of the accepted nodes, in
float64 and node by node.

openvino.genai PR #4847 (Fixes > Split validation windows) and optimum-intel PR #2098 (paged
attention targets) run these inside the target model and give no formulas; the definitions used on
both sides are written at each function. Requests are independent: every function takes one.
"""
import numpy as np


def tree_mask(parent, n, base=0):
    """(sees [T, T] bool, pos [T]): node i sees itself and its ancestors; pos = base + its ancestors' number.
    Nodes i >= n see nothing and have position 0; a parent that is not before its node makes it a root."""
    T = len(parent)
    sees, pos = np.zeros((T, T), bool), np.zeros(T, np.int64)
    for i in range(n):
        p = int(parent[i])
        if 0 <= p < i:
            sees[i] = sees[p]
            pos[i] = pos[p] + 1
        else:
            pos[i] = base
        sees[i, i] = True
    return sees, pos


def words(sees):
    """Bit j % 32 of word j // 32 of row i is sees[i, j]; int32 [T, W]."""
    T = sees.shape[-1]
    W = (T + 31) // 32
    out = np.zeros(sees.shape[:-1] + (W,), np.uint32)
    for j in range(T):
        out[..., j // 32] |= sees[..., j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def rope(x, cos, sin, interleaved):
    """x [..., D]; cos, sin [h] turn the first 2 h columns in pairs (f, f + h), or (2 f, 2 f + 1)."""
    x = np.array(x, np.float64)
    h = len(cos)
    a, b = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else (np.arange(h), np.arange(h, 2 * h))
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    x[..., a] = x1 * cos - x2 * sin
    x[..., b] = x2 * cos + x1 * sin
    return x


def attention(q, k, v, sees, scale, softcap=0.0):
    """q [T, Hq, D], k and v [S, H, D], sees [T, S] bool -> (out [T, Hq, D], lse [T, Hq], weighted magnitude
    sum_j p_j |v_j| [T, Hq, D], and [T, Hq] the largest scale * sum |q| |k| a row sees). A key that a row does
    not see is left out of its sums altogether; a row that sees nothing gives 0 and -inf."""
    T, Hq, D = q.shape
    H = k.shape[1]
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, big = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for i in range(T):
        at = np.flatnonzero(sees[i])
        if not len(at):
            continue
        for h in range(Hq):
            kk, vv, qq = k[at, h // (Hq // H)].astype(np.float64), v[at, h // (Hq // H)].astype(np.float64), q[i, h].astype(np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                x = kk @ qq * scale
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                m = x.max()
                p = np.exp(x - m)
                lse[i, h] = m + np.log(p.sum())
                p /= p.sum()
                out[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
                big[i, h] = scale * (np.abs(kk) @ np.abs(qq)).max()
    return out, lse, mag, big


def accept(tokens, parent, best, n):
    """(out_tokens [T], n_accepted, path [T]): from node 0 to the lowest child whose token is the choice at the
    node, until there is none; then the choice there. n = 0: -1 everywhere."""
    T = len(tokens)
    out, path = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    if n == 0:
        return out, -1, path
    cur, k = 0, 0
    path[0] = 0
    while True:
        nxt = [i for i in range(cur + 1, n) if parent[i] == cur and tokens[i] == best[cur]]
        if not nxt:
            out[k] = best[cur]
            return out, k, path
        cur = nxt[0]
        out[k] = tokens[cur]
        k += 1
        path[k] = cur


def commit(rows, ctx, path, n_accepted):
    """rows [slots, ...] of one request's cache; the accepted nodes' rows at slots ctx, ctx + 1, ..."""
    rows = rows.copy()
    old = rows.copy()
    for k in range(n_accepted + 1):
        rows[ctx + k] = old[ctx + path[k]]
    return rows
