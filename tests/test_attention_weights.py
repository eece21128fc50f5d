"""dt_tree_attention's weights at the ends of the types' ranges, against the
definition in 64 bits (pass_ref.py)."""

import numpy as np
import pytest
import torch

import pass_ref as ref
import test_verification_pass as tvp

bd = tvp.bd
BF16, F16 = torch.bfloat16, torch.float16


def sink_problem(keys, rows, heads, B, D, dtype, sink, low, high, seed):
    """One key with score 0 among `keys` whose scores (natural) lie between
    low and high for every query, the same for every request and head; values 1
    for all in the even elements, and -1 for the sink, 1 for the rest in the
    odd ones."""
    gen = torch.Generator().manual_seed(seed)
    score = low + (high - low) * torch.rand(keys, generator=gen)
    score[sink] = 0
    k = torch.zeros(keys, D)
    k[:, 0] = score * D ** 0.5 / 8
    v = torch.ones(keys, D)
    v[sink, 1::2] = -1
    q = torch.zeros(B, rows, heads, D)
    q[..., 0] = 8
    return q.to(dtype), k.to(dtype), v.to(dtype)


def shared_cache(k, v, P, heads, B, device, seed):
    """A cache whose requests share the pages (in random order) and whose heads
    share the elements: it is only read."""
    keys, D = k.shape
    pages = keys // P
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    pools = []
    for t in (k, v):
        back = torch.empty(pages, P, 1, D, dtype=t.dtype)
        back[order] = t.view(pages, P, 1, D)
        pools.append(back.to(device).expand(pages, P, heads, D))
    return bd.KVCache(pools[0], pools[1], order.to(torch.int32)[None].repeat(B, 1).to(device))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,D", [(1, 64), (1, 128), (1, 256), (40, 128), (70, 64), (70, 128), (70, 256)])
@pytest.mark.parametrize("low,high", [(-17.36, -17.36), (-21.0, -12.0)])
def test_many_small_weights_beside_a_large_one(device, dtype, rows, D, low, high):
    """The weights that a key with a far larger one leaves to the others are
    small each, but not together: 262144 of e^-17.36 make 0.75% of the sum.
    64 requests of 8 heads are so many that none is cut into chunks, each with
    a maximum of its own."""
    keys, B, heads = 262144, 64, 8
    print("[case] sink", dtype, rows, D, low, high, flush=True)
    for seed, sink in enumerate((0, keys // 2 + 11)):
        q, k, v = sink_problem(keys, rows, heads, B, D, dtype, sink, low, high, seed)
        kv = shared_cache(k, v, 64, heads, B, device, seed)
        got, lse = tvp.run_attention(device, [keys - rows] * B, rows, 0, None, None, q, kv, 0)
        K, V = k[:, :1].double().numpy(), v[:, :2].double().numpy()      # the others' products are zeros, and repeat
        for r in sorted({0, rows - 1}):
            n = keys - rows + r + 1
            want, wl, spread, slack, vmax = ref.attend_row(q[0, r, 0, :1].double().numpy(), K[:n], V[:n], D ** -0.5)
            # sums go by blocks of 16 keys and more; f16's weights, held 2^7 times as large, are off by half
            # of the type's smallest step below its normal range
            steps = keys // 16
            tol = ref.attend_tolerance(want, spread, slack, vmax, steps, dtype)
            if dtype == F16:
                tol = tol + n * ref.SMALLEST[F16] * 2.0 ** -7 * vmax
            err = np.abs(got[:, r].reshape(-1, 2) - want)
            assert np.all(err <= tol), (sink, r, err.max(0), tol)
            assert np.all(np.abs(lse[:, r] - wl) <= slack + ref.U32 * (4 * abs(wl) + steps + 16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,D", [(1, 64), (1, 128), (1, 256), (40, 128), (70, 64), (70, 128), (70, 256)])
def test_scores_far_from_zero_stay_finite(device, dtype, rows, D):
    """Scores of up to 2^27 that grow by a few units from tile to tile: their
    last bits are whole units, so the weights can only be told to be weights,
    and the result a mean of the values."""
    keys, heads, B, P = 3000, 1, 1, 16
    print("[case] far scores", dtype, rows, D, flush=True)
    gen = torch.Generator().manual_seed(rows + D)
    for far in (19, 22, 24, 25, 26, 27):
        for step in (0.02, 0.09, 0.3):
            k = torch.zeros(keys + rows, D)
            k[:, 0] = 2.0 ** (far - 13)
            k[:, 1] = step * torch.arange(keys + rows) * (1 + 0.3 * torch.rand(keys + rows, generator=gen))
            v = 1 + torch.rand(keys + rows, D, generator=gen)
            q = torch.zeros(B, rows, heads, D)
            q[..., 0], q[..., 1] = 2.0 ** 13, 1
            pad = -(keys + rows) % P
            k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).to(dtype) for t in (k, v))
            kv = shared_cache(k, v, P, heads, B, device, far)
            got, lse = tvp.run_attention(device, [keys], rows, 0, None, None, q.to(dtype), kv, 0, scale=1.0)
            # the weights' rounding beside their unrounded sum, twice, and the result's own
            slack = 4 * ref.HALF_STEP[dtype]
            assert np.all(np.isfinite(lse)), (far, step)
            assert np.all((got >= 1 - 2 * slack) & (got <= 2 + 2 * slack)), (far, step, got.min(), got.max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,D", [(1, 64), (1, 128), (1, 256), (40, 128), (70, 64), (70, 128), (70, 256)])
def test_seen_infinities_reach_a_row_times_their_weight(device, dtype, rows, D):
    """An infinity in v is the same in a tile that every query sees in full and
    in one that has unseen keys: infinite, and NaN where the weight is 0."""
    print("[case] seen infinities", dtype, rows, D, flush=True)
    keys, P, lead = 250, 16, 1
    seen = np.tril(np.ones((1, rows - 1, rows - 1), bool)) if rows > 1 else None
    # scores of the infinity's key, all others 0: e^-20 is 2^-29, still a weight in f16 (lifted to 2^-22),
    # e^-28 = 2^-40 is not, e^-120 = 2^-173 in neither type
    for score, weight in ((-5.0, True), (-20.0, True), (-28.0, dtype == BF16), (-120.0, False)):
        for at in (100, keys):                                    # in a whole tile; the chunk's first row
            k = torch.zeros(keys + rows, D)
            k[at, 0] = score * D ** 0.5 / 8
            v = torch.ones(keys + rows, D)
            v[at, 3], v[at, 4] = np.inf, -np.inf
            q = torch.zeros(1, rows, 1, D)
            q[..., 0] = 8
            pad = -(keys + rows) % P
            k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).to(dtype) for t in (k, v))
            kv = shared_cache(k, v, P, 1, 1, device, 5)
            got, lse = tvp.run_attention(device, [keys], lead, rows - 1, None, seen, q.to(dtype), kv, 0)
            assert np.all(np.isfinite(lse)), (score, at)
            want = (np.inf, -np.inf) if weight else (np.nan, np.nan)
            for x, w in zip((3, 4), want):
                col = got[0, :, 0, x]
                assert np.all(np.isnan(col)) if np.isnan(w) else np.all(col == w), (score, at, x, col)
            rest = [x for x in range(D) if x not in (3, 4)]
            # ones all: the weights' rounding beside their unrounded sum
            assert np.all(np.abs(got[0, :, 0][:, rest] - 1) <= 4 * ref.HALF_STEP[dtype]), (score, at)
