"""How dt_tree_attention cuts its work: the rule in exact terms (no GPU), and
calls with so much work for each resident workgroup that the chunk's size is
searched for, against the definition in 64 bits (pass_ref.py)."""

import ctypes

import numpy as np
import pytest
import torch

import pass_ref as ref

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

BF16, F16 = torch.bfloat16, torch.float16
UNIT, CUS, PLAN_BYTES = 64, 256, 256
MOST = 2 ** 30 // UNIT                                           # units of the longest segment there can be
f32 = np.float32


def shape_of(rows, G, D):
    """Rows of a tile, and workgroups resident at a time."""
    m = rows * G
    mt = 32 if m <= 32 else (64 if m <= 64 else 128)
    return mt, CUS * (2 if D == 64 else 1) if mt == 32 else CUS * (1 if D == 256 else 2)


def plan(ctx, live, rows, G, Hkv, D, cap):
    """(units of a chunk, whether its size was searched for, rounds, chunks,
    partial results) of a call, as the kernel derives them on the device."""
    mt, slots = shape_of(rows, G, D)
    requests = [(n, -(-n * G // mt), -(-min(c + n, cap) // UNIT)) if c >= 0 else (0, 0, 0) for c, n in zip(ctx, live)]
    work = float(sum(m * Hkv * u for _, m, u in requests))
    segs, longest = sum(m * Hkv for _, m, _ in requests), max(u for _, _, u in requests)
    each = f32(work) / f32(slots)
    searched = not (each < 16 or len(ctx) > 512)
    if not searched:
        room = slots - segs if 2 * segs < slots else slots
        c = max(4, int(min(f32(work) / f32(room), f32(MOST))) + 1)
    else:
        best = None
        for lane in range(64):
            want = min(each * f32(1 + 0.0625 * (lane & 15)) / f32(1 + (lane >> 4)), f32(MOST))
            size = max(4, longest if lane == 0 else int(want) + 1)
            inv = f32(1) / f32(size)
            jobs = sum(m * Hkv * int(f32(u + size - 1) * inv) for _, m, u in requests)
            cost = f32(-(-jobs // slots)) * (f32(min(longest, size)) + f32(4 if longest > size else 0))
            if best is None or (cost, -size) < best:
                best = (cost, -size)
        c = -best[1]
    chunks = sum(m * Hkv * -(-u // c) for n, m, u in requests if n)
    partials = sum(m * Hkv * -(-u // c) for n, m, u in requests if -(-u // c) > 1)
    return c, searched, -(-chunks // slots), chunks, partials, slots, mt


def workspace_partials(B, lead, n_max, G, Hkv, D):
    """Partial results that dt_attention_workspace() has room for."""
    kv = bd._KVCache(k=1 << 20, v=1 << 20, page_table=1 << 20, page_stride=1 << 20, slot_stride=1 << 14,
                     head_stride=1 << 8, layers=1, num_pages=2, page_size=16, max_pages=8, Hkv=Hkv, D=D, dtype=1)
    chunk = bd._Chunk(B=B, lead=lead, n_max=n_max)
    n = bd._load().dt_attention_workspace(ctypes.byref(kv), ctypes.byref(chunk), G * Hkv)
    mt = shape_of(lead + n_max, G, D)[0]
    return (n - PLAN_BYTES) // (mt * (D + 2) * 4)


@pytest.mark.parametrize("seed", range(12))
def test_partial_results_fit_the_workspace(seed):
    """Batches of all kinds of lengths: no more partial results, and no more
    chunks, than the caller's workspace and the launched grid hold."""
    rs = np.random.RandomState(seed)
    searches = 0
    for _ in range(60):
        B = int(2 ** rs.uniform(0, 9.5))
        rows = int(2 ** rs.uniform(0, 12))
        G, Hkv, D = int(rs.randint(1, 9)), int(rs.choice([1, 2, 4, 8])), int(rs.choice([64, 128, 256]))
        top = 2 ** rs.uniform(0, 21)
        kind = rs.randint(3)
        ctx = [int(top * (x if kind == 0 else (x ** 6 if kind == 1 else 1))) for x in rs.rand(B)]
        live = [int(n) for n in rs.randint(1, rows + 1, B)]
        c, searched, _, chunks, partials, slots, mt = plan(ctx, live, rows, G, Hkv, D, 1 << 30)
        searches += searched
        segments = B * Hkv * -(-rows * G // mt)
        assert chunks <= segments + 4 * slots
        assert partials <= workspace_partials(B, 1, rows - 1, G, Hkv, D), (ctx[:4], rows, G, Hkv, D, c)
    assert searches > 10


@pytest.mark.parametrize("B,rows,G,Hkv,keys", [(1, 65536, 2048, 1, 2 ** 30), (255, 65536, 1, 64, 2 ** 30 - 1),
                                               (4096, 4096, 127, 1, 2 ** 30), (2048, 8192, 4, 16, 2 ** 29)])
def test_chunks_of_the_most_work_there_can_be(B, rows, G, Hkv, keys):
    """The largest calls that dt.h admits: a share of a slot passes 2^31 units,
    a chunk's size does not, and nothing is cut below the workspace."""
    assert B * rows <= 2 ** 24 and B * rows * G * Hkv < 2 ** 31
    c, _, _, chunks, partials, slots, mt = plan([keys - rows] * B, [rows] * B, rows, G, Hkv, 128, 2 ** 30)
    assert 4 <= c <= MOST + 1
    assert chunks <= B * Hkv * -(-rows * G // mt) + 4 * slots
    assert partials <= workspace_partials(B, 0, rows, G, Hkv, 128)


CASES = {
    # ctx (lowest, highest), B, lead, n_max, nodes (lowest), mask, G, Hkv, D, page, type
    "decode, more requests than lanes": ((33, 16383), 80, 1, 0, 0, None, 4, 8, 128, 16, BF16),
    "decode, heads of 64": ((1, 9001), 130, 1, 0, 0, None, 7, 4, 64, 20, F16),
    "decode, heads of 256": ((100, 7000), 65, 1, 0, 0, None, 5, 4, 256, 16, BF16),
    "one request, a million keys": ((1000000, 1000000), 1, 1, 0, 0, None, 8, 1, 128, 256, F16),
    "two draft rows a request": ((0, 12000), 70, 1, 15, 3, "tree", 3, 8, 128, 20, F16),
    "trees": ((500, 9000), 70, 1, 64, 40, "tree", 4, 4, 128, 16, BF16),
    "trees, heads of 64": ((10, 9000), 66, 3, 200, 100, "tree", 7, 2, 64, 32, F16),
    "trees, heads of 256": ((3000, 4000), 33, 1, 40, 38, "tree", 4, 4, 256, 24, BF16),
    "small trees, heads of 256": ((30, 6000), 70, 1, 11, 8, "tree", 4, 4, 256, 16, F16),
    "prompt chunks": ((4001, 9000), 2, 0, 2048, 1801, None, 4, 4, 128, 64, BF16),
    "prompt chunks, one of them short": ((3, 20000), 3, 0, 700, 1, None, 5, 3, 64, 16, F16),
    "prompt chunks, heads of 256": ((2000, 3000), 3, 0, 1000, 900, None, 2, 4, 256, 1, F16),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_searched_splits(device, name):
    (lo, hi), B, lead, n_max, nn_lo, kind, G, Hkv, D, P, dtype = CASES[name]
    rs = np.random.RandomState(len(name))
    rows, Hq = lead + n_max, G * Hkv
    spread = lambda a, b: [int(x) for x in rs.permutation(np.linspace(a, b, B).astype(int))] if B > 1 else [b]  # noqa: E731
    ctx, nn = spread(lo, hi), spread(nn_lo, n_max)
    if B > 9:
        ctx[5] = -1                                               # a request without rows
    live = [lead + n if c >= 0 else 0 for c, n in zip(ctx, nn)]
    # requests share the pages of a small pool at random: attention only reads
    pages = 4096 // P + 7
    table = rs.randint(0, pages, (B, -(-(max(ctx) + rows) // P) + 3)).astype(np.int32)
    table[B - 1, 1] = pages                                       # a page that is not there
    c, searched, rounds, chunks, partials, slots, mt = plan(ctx, live, rows, G, Hkv, D, table.shape[1] * P)
    print(f"[case] {name}: chunks of {c} units, {chunks} over {slots} slots, {partials} partial results", flush=True)
    assert searched
    gen = torch.Generator().manual_seed(len(name))
    k, v = (torch.randn(pages, P, Hkv, D, generator=gen).to(dtype) for _ in range(2))
    q = torch.randn(B, rows, Hq, D, generator=gen).to(dtype)
    seen = ref.random_tree(rs, B, n_max, nn, width=8)[2] if kind else None
    i32 = dict(dtype=torch.int32, device=device)
    kv = bd.KVCache(k.to(device), v.to(device), torch.from_numpy(table).to(device))
    chunk = bd.Chunk(torch.tensor(ctx, **i32), lead, n_max, torch.tensor(nn, **i32),
                     mask=torch.from_numpy(ref.pack_bits(seen)).to(device) if kind else None)
    need, guard = bd.dt_attention_workspace(kv, chunk, Hq), 1 << 16
    ws = torch.full((need + 2 * guard,), 255, dtype=torch.uint8, device=device)
    dq, out = q.to(device), torch.full(q.shape, 7.0, dtype=dtype, device=device)
    lse = torch.full(q.shape[:3], 7.0, device=device)
    bd.dt_tree_attention(kv, chunk, dq, out, lse=lse, workspace=ws[guard:guard + need])
    torch.cuda.synchronize()
    assert bool((ws[:guard] == 255).all()) and bool((ws[guard + need:] == 255).all()), "outside of the workspace"
    assert int(ws[guard:guard + 4].view(torch.int32)) == c
    got, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    order = np.argsort([x + y for x, y in zip(ctx, live)])
    sample = {int(order[-1]), int(order[B // 2]), int(order[0]), B - 1, min(B - 1, 63), min(B - 1, 64)}
    for b in range(B):
        assert np.all(got[b, live[b]:] == 7) and np.all(lse[b, live[b]:] == 7)
    K64, V64 = k.double().numpy(), v.double().numpy()
    for b in sorted(sample):
        if not live[b]:
            continue
        picks = {0, live[b] - 1, *rs.randint(0, live[b], 4).tolist()}
        for r in sorted(picks):
            slots_seen = np.array(ref.visible(ctx[b], lead, r, nn[b], None if seen is None or r < lead
                                              else seen[b, r - lead]))
            pg, off = table[b][slots_seen // P], slots_seen % P
            there = pg < pages
            pg, off = pg[there], off[there]
            # sums go by 16 keys and more, and join no more chunks than there are 256 keys
            steps = len(pg) // 16 + len(pg) // 256 + 64
            for h in {0, Hq - 1, int(rs.randint(Hq))}:
                want, wl, spr, slack, vmax = ref.attend_row(q[b, r, h].double().numpy(), K64[pg, off, h // G],
                                                            V64[pg, off, h // G], D ** -0.5)
                tol = ref.attend_tolerance(want, spr, slack, vmax, steps, dtype)
                if dtype == F16:                                  # weights below the normal range, one a key
                    tol = tol + len(pg) * ref.SMALLEST[F16] * 2.0 ** -7 * vmax
                err = np.abs(got[b, r, h] - want)
                assert np.all(err <= tol), (b, r, h, float((err - tol).max()))
                assert abs(lse[b, r, h] - wl) <= slack + ref.U32 * (4 * abs(wl) + steps + 16), (b, r, h)


@pytest.mark.gpu
def test_captured_calls_follow_their_lengths(device):
    """A captured call is replayed for lengths that were written after its
    capture, shorter and far longer ones: the split follows the device's values."""
    print("[case] captured lengths", flush=True)
    B, Hkv, G, D, P, lead, n_max = 5, 2, 4, 128, 16, 1, 30
    rs = np.random.RandomState(8)
    gen = torch.Generator(device=device).manual_seed(8)
    pages = 500
    k, v = (torch.empty(pages, P, Hkv, D, dtype=BF16, device=device).normal_(generator=gen) for _ in range(2))
    table = torch.from_numpy(rs.randint(0, pages, (B, 1300)).astype(np.int32)).to(device)
    i32 = dict(dtype=torch.int32, device=device)
    kv = bd.KVCache(k, v, table)
    seen = torch.from_numpy(ref.pack_bits(ref.random_tree(rs, B, n_max, [n_max] * B)[2])).to(device)
    chunk = bd.Chunk(torch.full((B,), 7, **i32), lead, n_max, torch.full((B,), 3, **i32), mask=seen)
    q = torch.empty(B, lead + n_max, Hkv * G, D, dtype=BF16, device=device).normal_(generator=gen)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device=device)
    ws = torch.empty(bd.dt_attention_workspace(kv, chunk, Hkv * G), dtype=torch.uint8, device=device)
    call = lambda: bd.dt_tree_attention(kv, chunk, q, out, lse=lse, workspace=ws)      # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for ctx, nn in (([0, 1, 2, 3, 4], [0, 30, 5, 1, 2]), ([20000, 9000, 300, 64, 15000], [30, 29, 0, 12, 30]),
                    ([7] * 5, [3] * 5), ([-1, 20000, -1, 2, 700], [30] * 5), ([12000] * 5, [17] * 5)):
        chunk.ctx_len.copy_(torch.tensor(ctx, **i32))
        chunk.n_nodes.copy_(torch.tensor(nn, **i32))
        results = []
        for run in (call, graph.replay, graph.replay):
            out.fill_(7)
            lse.fill_(7)
            run()
            torch.cuda.synchronize()
            results.append((out.clone(), lse.clone()))
        for o, s in results[1:]:
            assert torch.equal(o.view(torch.int16), results[0][0].view(torch.int16)) and torch.equal(s, results[0][1])
        for b in range(B):
            live = 0 if ctx[b] < 0 else lead + nn[b]
            assert bool((results[0][0][b, live:] == 7).all())
            assert bool(torch.isfinite(results[0][1][b, :live]).all())
            if live:                                              # the root row sees all slots up to its own
                n = ctx[b] + 1
                at = torch.arange(n, device=device)
                K, V = (t[table[b].long()[at // P], at % P].double().cpu().numpy() for t in (k, v))
                want, wl, spr, slack, vmax = ref.attend_row(q[b, 0, 0].double().cpu().numpy(), K[:, 0], V[:, 0],
                                                            D ** -0.5)
                steps = n // 16 + n // 256 + 64
                tol = ref.attend_tolerance(want, spr, slack, vmax, steps, BF16)
                assert np.all(np.abs(results[0][0][b, 0, 0].double().cpu().numpy() - want) <= tol)
                assert abs(float(results[0][1][b, 0, 0]) - wl) <= slack + ref.U32 * (4 * abs(wl) + steps + 16)
