"""Latent attention and drawn tokens from their definitions (dt.h), in 64-bit
arithmetic on the CPU; and problems of all kinds for them.  Shares no code with
the library."""

import math

import numpy as np
import torch

from pass_ref import HALF_STEP, SMALLEST, U32, pack_bits, random_tree, rows_of, slot_at


def make_latents(rs, ctx, rows, P, D, dtype, layers=1, spare=3, width=0, sd=1.0):
    """Random pages in random order; -1 behind a request's last page.  Unused
    slots hold NaN."""
    need = [max((max(c, 0) + rows + P - 1) // P, 1) for c in ctx]
    pages = sum(need) + spare
    order = rs.permutation(pages).astype(np.int32)
    table = np.full((len(ctx), max(need + [width])), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    c = torch.from_numpy(rs.standard_normal((layers, pages, P, D)) * sd).to(dtype)
    used = np.zeros((pages, P), bool)
    for b, n in enumerate(ctx):
        for s in range(max(n, 0)):
            used[table[b, s // P], s % P] = True
    c[:, torch.from_numpy(~used)] = math.nan
    return c, table


def fill_chunk(rs, c, table, ctx, rows, sd=1.0):
    """Finite latents in the chunk's own slots (as an append leaves them)."""
    P = c.shape[2]
    for b, n in enumerate(ctx):
        for s in range(max(n, 0), max(n, 0) + rows):
            at = slot_at(table, c.shape[1], P, b, s)
            if n >= 0 and at is not None:
                c[:, at[0], at[1]] = torch.from_numpy(rs.standard_normal(c.shape[-1]) * sd).to(c.dtype)


def seen_slots(table, num_pages, P, b, ctx, lead, r, nn, seen_row, cap):
    """Slots that row r sees, without those the cache does not have."""
    if r < lead or seen_row is None:
        slots = list(range(ctx + r + 1))
    else:
        slots = list(range(ctx + lead)) + [ctx + lead + j for j in range(nn) if seen_row[j]]
    return [s for s in slots if s < cap and slot_at(table, num_pages, P, b, s) is not None]


def attend(q, K, V, scale, dtype, score_error=0.0, value_error=0.0):
    """Queries [Hq, D] over keys [S, D] and values [S, N] of each head (or of
    all: [D, S] shared): (out [Hq, N], lse, tolerance).  score_error: what the
    keys' roundings move a score by, per head; value_error: relative one of the
    values."""
    Hq = q.shape[0]
    if K.shape[-2] == 0:
        n = V.shape[-1]
        return np.zeros((Hq, n)), np.full(Hq, -math.inf), np.zeros((Hq, n)) + SMALLEST[dtype], np.zeros(Hq)
    x = scale * np.einsum("hd,hsd->hs", q, np.broadcast_to(K, (Hq,) + K.shape[-2:]))
    top = x.max(1, keepdims=True)
    p = np.exp(x - top)
    total = p.sum(1, keepdims=True)
    p /= total
    Vb = np.broadcast_to(V, (Hq,) + V.shape[-2:])
    out, spread = np.einsum("hs,hsn->hn", p, Vb), np.einsum("hs,hsn->hn", p, np.abs(Vb))
    size = np.einsum("hd,hsd->hs", np.abs(q), np.abs(np.broadcast_to(K, (Hq,) + K.shape[-2:]))).max(1)
    # fp32 score: D products in any order, scaled, the maximum subtracted, put through exp2
    slack = U32 * ((q.shape[1] + 4) * scale * size + 4 * np.abs(x).max(1) + 8) + score_error
    # half a step of the result; each weight half a step and its score's error, its sum again; weights
    # below the type's normal range, half its smallest step each; fp32 sums, rescaled at most once a tile;
    # the values' own roundings
    S = x.shape[1]
    per = HALF_STEP[dtype] + 2 * slack + U32 * (S + 64) + value_error
    tol = (HALF_STEP[dtype] * np.abs(out) + per[:, None] * spread * (1 + HALF_STEP[dtype]) +
           S * SMALLEST[dtype] * (np.abs(Vb).max((1, 2)) / total[:, 0])[:, None] + SMALLEST[dtype])
    return out, (top + np.log(total))[:, 0], tol, slack


def draw_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, distance) of one row of logits: `distance` is how near u
    comes to where another token would be drawn, and a sum to where another
    token would stay, relative to the sum of the weights."""
    x = np.asarray(x, np.float64)
    best = int(np.argmax(x))
    if x[best] == -np.inf:
        return -1, -np.inf, 1.0
    if not temperature > 0:
        return best, 0.0, 1.0
    order = np.argsort(-x, kind="stable")
    if 0 < top_k < len(order):
        order = order[:top_k]
    w = np.exp((x[order] - x[best]) / temperature)
    near = 1.0
    stay = np.ones(len(w), bool)
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        limit = top_p * math.fsum(w)
        stay &= before < limit
        gap = np.abs(before - limit)[1:]
        near = min(near, float(gap.min()) / w.sum()) if len(gap) else near
    if min_p > 0:
        stay &= w >= min_p
        gap = np.abs(w - min_p)[w < 1]
        near = min(near, float(gap.min())) if len(gap) else near
    stay[0] = True
    kept = np.sort(order[stay])
    w = np.exp((x[kept] - x[best]) / temperature)
    upto = np.cumsum(w)
    target = float(u) * upto[-1]
    i = min(int(np.searchsorted(upto, target, side="right")), len(kept) - 1)
    near = min(near, float(np.abs(upto[:-1] - target).min()) / upto[-1]) if len(kept) > 1 else near
    return int(kept[i]), math.log(w[i] / upto[-1]) if w[i] > 0 else -math.inf, near
