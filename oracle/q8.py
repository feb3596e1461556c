"""The cache in 8 bits and sampled acceptance along a tree (oracle; test infrastructure only).

openvino.genai PR #4847 (commit on exact sampled speculative decoding) gives the acceptance rule for one draft after the other;
the format is that of dspark.h: blocks of 32 columns share a power of two, codes are e4m3 or whole numbers.
"""
import numpy as np

# the numbers of e4m3's codes 0..127, from the format: 4 exponent bits (bias 7), 3 fraction bits, no infinities (0x7F is no number; 480 here)
E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(128)])


def turn(x, cos, sin, interleaved):
    """oracle.tree.rope in float32, every product and every sum rounded by itself."""
    x = np.array(x, np.float32)
    cos, sin = np.asarray(cos, np.float32), np.asarray(sin, np.float32)
    h = len(cos)
    a, b = (np.arange(0, 2 * h, 2), np.arange(1, 2 * h, 2)) if interleaved else (np.arange(h), np.arange(h, 2 * h))
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    x[..., a] = x1 * cos - x2 * sin
    x[..., b] = x2 * cos + x1 * sin
    return x


def quantise_block(y, e4m3):
    """(codes uint8, scale byte) of one block of float32 numbers."""
    y = np.asarray(y, np.float64)
    most = 448.0 if e4m3 else 127.0
    m = np.abs(y[np.isfinite(y)]).max(initial=0.0)
    e = -126
    while e < 118 and m > most * 2.0 ** e:
        e += 1
    with np.errstate(invalid="ignore"):
        z = np.clip(np.where(np.isnan(y), 0.0, y) * 2.0 ** -e, -most, most)
    if not e4m3:
        return np.rint(z).astype(np.int8).view(np.uint8), e + 127
    low = np.searchsorted(E4M3, np.abs(z), side="right") - 1                 # the code at or below, then ties to the even code
    up = np.minimum(low + 1, 126)
    d0, d1 = np.abs(z) - E4M3[low], E4M3[up] - np.abs(z)
    code = np.where((d1 < d0) | ((d1 == d0) & (low % 2 == 1) & (up > low)), up, low)
    return (code | np.where(np.signbit(z), 128, 0)).astype(np.uint8), e + 127


def quantise(y, e4m3):
    """y [..., D] float32 -> (codes [..., D] uint8, scale bytes [..., blocks] uint8)."""
    D = y.shape[-1]
    codes, scale = np.zeros(y.shape, np.uint8), np.zeros(y.shape[:-1] + ((D + 31) // 32,), np.uint8)
    for at in np.ndindex(*y.shape[:-1]):
        for b in range(scale.shape[-1]):
            codes[at][32 * b:32 * b + 32], scale[at][b] = quantise_block(y[at][32 * b:32 * b + 32], e4m3)
    return codes, scale


def numbers(codes, scale, e4m3):
    """What codes [..., D] and scale bytes [..., blocks] (uint8) stand for, in float64."""
    c = np.where(codes & 128, -1.0, 1.0) * E4M3[codes & 127] if e4m3 else codes.view(np.int8).astype(np.float64)
    p = 2.0 ** (np.clip(scale.astype(np.float64), 1, 245) - 127)
    return c * np.repeat(p, 32, -1)[..., :codes.shape[-1]]


def residual(p, q, a, refused):
    """max(0, p - a q) in float64, or p without the refused tokens."""
    if q is not None:
        return np.maximum(0.0, p.astype(np.float64) - a * q.astype(np.float64))
    rho = p.astype(np.float64)
    rho[list(refused)] = 0.0
    return rho


def pick(rho, u):
    """First index at which the running sum passes u times the total; the last above 0 if none does."""
    run = np.cumsum(rho)
    at = np.flatnonzero((run > u * run[-1]) & (rho > 0))
    return int(at[0]) if len(at) else int(np.flatnonzero(rho > 0)[-1])


def verify(p, q, tokens, parent, n, u_accept, u_draw):
    """(out_tokens [T], n_accepted, path [T]) of one request, child by child with the whole residual."""
    T = len(tokens)
    out, path = np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    if n == 0:
        return out, -1, path
    cur, k = 0, 0
    path[0] = 0
    while True:
        a, b, refused, gone = 0.0, 1.0, set(), False
        for x in range(cur + 1, n):
            if parent[x] != cur:
                continue
            t = int(tokens[x])
            if not 0 <= t < p.shape[1]:
                continue
            rho = residual(p[cur], None if q is None else q[cur], a, refused)
            if u_accept[x] * b * (1.0 if q is None else float(q[cur, t])) < rho[t]:
                out[k] = t
                k += 1
                path[k] = cur = x
                gone = True
                break
            if q is None:
                b -= rho[t]
                refused.add(t)
            else:
                a += b
                b = residual(p[cur], q[cur], a, refused).sum()
        if gone:
            continue
        rho = residual(p[cur], None if q is None else q[cur], a, refused)
        if not rho.sum() > 0:
            rho = p[cur].astype(np.float64)
        out[k] = pick(rho, u_draw) if 0 < rho.sum() < np.inf else -1
        return out, k, path
