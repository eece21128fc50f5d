"""The verification pass's operators from their definitions (dt.h), in 64-bit
arithmetic on the CPU, one request, row and head at a time; and problems of
all kinds for them.  Shares no code with the library."""

import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # relative
SMALLEST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half a subnormal step
U32 = 2.0 ** -24


def pack_bits(seen: np.ndarray) -> np.ndarray:
    """[..., n] truth values -> [..., ceil(n/32)] int32, lowest index in the lowest bit."""
    n = seen.shape[-1]
    words = (n + 31) // 32
    full = np.zeros(seen.shape[:-1] + (words * 32,), bool)
    full[..., :n] = seen
    return np.packbits(full, axis=-1, bitorder="little").view(np.int32).reshape(seen.shape[:-1] + (words,))


def random_tree(rs, B, n_max, n_nodes, width=4):
    """BFS-ordered random trees: tokens, parents, depths, ancestor truth values."""
    parents = np.full((B, n_max), -1, np.int32)
    depths = np.zeros((B, n_max), np.int32)
    seen = np.zeros((B, n_max, n_max), bool)
    for b in range(B):
        for i in range(n_nodes[b]):
            t = i // width
            depths[b, i] = t + 1
            if t:
                parents[b, i] = (t - 1) * width + rs.randint(width)
                seen[b, i] = seen[b, parents[b, i]]
            seen[b, i, i] = True
    return parents, depths, seen


def rows_of(b, ctx, lead, n_max, n_nodes):
    if ctx[b] < 0:
        return 0
    n = n_max if n_nodes is None else min(max(int(n_nodes[b]), 0), n_max)
    return lead + n


def slot_at(table, num_pages, P, b, slot):
    """(page, offset) of a slot, or None where the cache has no such token."""
    if slot // P >= table.shape[1]:
        return None
    page = int(table[b, slot // P])
    return (page, slot % P) if 0 <= page < num_pages else None


# ---------------------------------------------------------------------------

def append_head(x, w, eps, pos, freqs, interleaved, rot_scale):
    """One head (float64 [D]) normed and turned; also the size of each
    element's pair, which bounds the rounding of a difference."""
    x = np.array(x, np.float64)
    if w is not None:
        x = x / math.sqrt(float(np.mean(x * x)) + eps) * w
    y, size = x.copy(), np.abs(x)
    half = 0 if freqs is None else len(freqs)
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = x[lo], x[hi]
        c, s = math.cos(pos * freqs[i]) * rot_scale, math.sin(pos * freqs[i]) * rot_scale
        y[lo], y[hi] = a * c - b * s, a * s + b * c
        size[lo] = size[hi] = math.hypot(a, b) * abs(rot_scale)
    return y, size


def append_tolerance(want, size, dtype):
    """Half a step of the result, and 48 fp32 roundings of the pair: up to 16
    in the sum of squares (8 in a lane, then a tree), the square root and two
    products (5), the angle (pi) and its sine and cosine (4 each), the turn
    (3), with some to spare."""
    return HALF_STEP[dtype] * np.abs(want) + 48 * U32 * size * (1 + HALF_STEP[dtype]) + SMALLEST[dtype]


def visible(ctx, lead, r, nn, seen_row):
    """Slots that row r sees, as a list."""
    if r < lead or seen_row is None:
        return list(range(ctx + r + 1))
    return list(range(ctx + lead)) + [ctx + lead + j for j in range(nn) if seen_row[j]]


def attend_row(q, K, V, scale):
    """One query (float64 [D]) over the keys it sees: (out, lse, tolerance
    parts).  spread = sum p |v|; slack = bound on the error of a score."""
    D = q.shape[0]
    if K.shape[0] == 0:
        return np.zeros(D), -math.inf, np.zeros(D), 0.0, 0.0
    x = scale * (K @ q)
    top = x.max()
    p = np.exp(x - top)
    total = p.sum()
    # fp32 score: D products added in any order, then scaled, the maximum
    # subtracted and put through exp2 (argument and function)
    slack = U32 * ((D + 4) * scale * float((np.abs(K) @ np.abs(q)).max()) + 4 * float(np.abs(x).max()) + 8)
    return p @ V / total, top + math.log(total), p @ np.abs(V) / total, slack, float(np.abs(V).max()) / total


def attend_tolerance(want, spread, slack, vmax, keys, dtype):
    """Half a step of the result; each weight half a step and the error of
    its score, its sum again; weights below the type's normal range, off by at
    most half its smallest step, one a key; fp32 sums of the products, rescaled
    at most once a tile."""
    per_weight = HALF_STEP[dtype] + 2 * slack + U32 * (keys + 64)
    return (HALF_STEP[dtype] * np.abs(want) + per_weight * spread * (1 + HALF_STEP[dtype]) +
            keys * SMALLEST[dtype] * vmax + SMALLEST[dtype])


def logits_row(x, count, prompt, rep, freq, pres, bias, allowed):
    """(want, size of the largest step, touched) of one row, float64 [V]."""
    x = x.astype(np.float64)
    seen = (count > 0) | prompt
    y = np.where(seen, np.where(x > 0, x / rep, x * rep), x)
    size = np.where(np.isfinite(x), np.abs(y), 0)
    cost = freq * count + pres * (count > 0)
    y = y - cost
    touched = seen | (bias != 0)
    size = size + np.abs(freq) * count + np.abs(pres) + np.where(np.isfinite(bias), np.abs(bias), 0)
    y = np.where(bias != 0, y + bias, y)
    if allowed is not None:
        y = np.where(allowed, y, -np.inf)
        touched = touched & allowed
    return y, size, touched


def walk(tokens, parents, target, lead, nn, L):
    """(accepted tokens and the target's next, accepted nodes) of one tree."""
    cur, nodes, said = -1, [], []
    while True:
        want = int(target[lead + cur])
        said.append(want)
        kids = [i for i in range(cur + 1, nn) if parents[i] == cur and tokens[i] == want]
        if not kids or len(nodes) == L - 1:
            return said, nodes
        cur = kids[0]
        nodes.append(cur)
