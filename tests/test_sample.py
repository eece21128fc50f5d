"""dt_sample_rows against its definition in 64 bits (latent_ref.draw_row)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import latent_ref as lat
import pass_ref as ref

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BAD, LIMIT, WORK = bd.DT_ERR_INVALID_ARG, bd.DT_ERR_UNSUPPORTED, bd.DT_ERR_WORKSPACE
FAKE = 0x100000
NOT_DRAWN = -77


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# refusals (no GPU)
# ---------------------------------------------------------------------------

def _params(**kw):
    p = bd._SampleParams()
    for k, v in dict(dict(logits=FAKE, B=2, lead=1, n_max=3, V=1000, dtype=1, u=FAKE, tokens=FAKE, workspace=FAKE,
                          workspace_bytes=1 << 40), **kw).items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), BAD), (dict(logits=FAKE + 8), BAD), (dict(B=-1), BAD), (dict(lead=-1), BAD), (dict(n_max=-1), BAD),
    (dict(lead=0, n_max=0), BAD), (dict(V=0), BAD), (dict(dtype=2), BAD), (dict(dtype=-1), BAD), (dict(u=None), BAD),
    (dict(tokens=None), BAD), (dict(u=FAKE + 2), BAD), (dict(tokens=FAKE + 1), BAD), (dict(logp=FAKE + 2), BAD),
    (dict(n_nodes=FAKE + 2), BAD), (dict(temperature=FAKE + 2), BAD), (dict(top_k=FAKE + 1), BAD),
    (dict(top_p=FAKE + 3), BAD), (dict(min_p=FAKE + 2), BAD), (dict(B=65536), LIMIT), (dict(lead=65536), LIMIT),
    (dict(B=4096, n_max=4096), LIMIT), (dict(V=1 << 26), LIMIT), (dict(workspace=FAKE + 8), WORK),
    (dict(workspace=None), WORK), (dict(workspace_bytes=0), WORK),
])
def test_refusals(kw, status):
    if status == WORK:                                            # a call that needs some
        kw = dict(dict(B=1, n_max=0, V=100000), **kw)
        if bd._load().dt_sample_workspace(ctypes.byref(_params(B=1, n_max=0, V=100000))) == 0:
            return
    assert bd._load().dt_sample_rows(ctypes.byref(_params(**kw))) == status


def test_empty_batches_null_and_workspace():
    lib = bd._load()
    assert lib.dt_sample_rows(None) == BAD
    assert lib.dt_sample_rows(ctypes.byref(_params(B=0, logits=None, u=None, tokens=None, workspace=None))) == bd.DT_OK
    assert lib.dt_sample_workspace(None) == 0
    assert lib.dt_sample_workspace(ctypes.byref(_params(V=0))) == 0
    x = torch.zeros(0, 3, 50)
    bd.dt_sample_rows(x, torch.zeros(0, 3), torch.zeros(0, 3, dtype=I32))


@pytest.mark.parametrize("dtype,V", [(0, 1), (0, 32000), (1, 151936), (1, (1 << 26) - 1)])
def test_no_call_needs_a_workspace(dtype, V):
    assert bd._load().dt_sample_workspace(ctypes.byref(_params(dtype=dtype, V=V, B=1, n_max=0))) == 0
    assert bd.dt_sample_workspace(torch.empty(2, 3, V, dtype=(F32, BF16)[dtype], device="meta")) == 0


def test_binding_checks_tensors():
    x, u, t = torch.zeros(2, 3, 50), torch.zeros(2, 3), torch.zeros(2, 3, dtype=I32)
    for bad in (dict(logits=x.half()), dict(logits=x[0]), dict(logits=x[..., ::2]), dict(u=u[:1]), dict(u=u.double()),
                dict(tokens=t.long()), dict(tokens=t[:, :2]), dict(temperature=torch.zeros(3)), dict(top_k=torch.zeros(2)),
                dict(top_p=torch.zeros(2, dtype=torch.float64)), dict(min_p=torch.zeros(2, 1)), dict(logp=u.double()),
                dict(lead=4), dict(lead=-1), dict(n_nodes=torch.zeros(2))):
        with pytest.raises(bd.DtError):
            bd.dt_sample_rows(**dict(dict(logits=x, u=u, tokens=t), **bad))
    with pytest.raises(bd.DtError, match="must be on a GPU"):
        bd.dt_sample_rows(x, u, t)
    with pytest.raises(bd.DtError):
        bd.dt_sample_workspace(x[0])


def test_the_definition_on_a_row_done_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 4.0, 1.0]))               # of 12
    for u, want in ((0.0, 0), (0.08, 0), (0.084, 1), (0.41, 1), (0.42, 2), (0.58, 2), (0.59, 3), (0.92, 4), (0.99, 4)):
        assert lat.draw_row(x, u)[0] == want
    assert [lat.draw_row(x, u, top_k=2)[0] for u in (0, 0.49, 0.51, 0.99)] == [1, 1, 3, 3]
    assert [lat.draw_row(x, u, top_k=1)[0] for u in (0, 0.99)] == [1, 1]
    assert [lat.draw_row(x, u, top_p=0.3)[0] for u in (0, 0.99)] == [1, 1]
    assert [lat.draw_row(x, u, top_p=0.4)[0] for u in (0, 0.99)] == [1, 3]
    assert [lat.draw_row(x, u, min_p=0.4)[0] for u in (0, 0.41, 0.61, 0.99)] == [1, 2, 3, 3]
    assert lat.draw_row(x, 0.5, temperature=0.0)[:2] == (1, 0.0)
    assert lat.draw_row(np.full(3, -np.inf), 0.5)[0] == -1


# ---------------------------------------------------------------------------

def draw(device, x, u, nn=None, lead=None, stream=None, **how):
    """Tokens and logp of logits [B][rows][V]; how: lists of a value a request."""
    B, rows, V = x.shape
    kinds = dict(temperature=F32, top_k=I32, top_p=F32, min_p=F32)
    how = {k: torch.tensor(v, dtype=kinds[k], device=device) for k, v in how.items()}
    dx = x.to(device)
    tokens = torch.full((B, rows), NOT_DRAWN, dtype=I32, device=device)
    logp = torch.full((B, rows), 9.0, device=device)
    need = bd.dt_sample_workspace(dx)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=device) if need else None
    bd.dt_sample_rows(dx, u.to(device), tokens, logp=logp, lead=lead, workspace=ws, stream=stream,
                      n_nodes=None if nn is None else torch.tensor(nn, dtype=I32, device=device), **how)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), logp.cpu().numpy()


def check(x, u, tokens, logp, nn=None, lead=None, **how):
    """Tokens equal wherever no border lies within the documented rounding of
    the weights of u and the limits: V weights, off by half of 2^(n - 62) and
    2^-43 of themselves each, against a sum of one at least."""
    B, rows, V = x.shape
    lead = rows if lead is None else lead
    room = V * (2.0 ** (math.ceil(math.log2(max(V, 2))) - 62) + 2.0 ** -43)
    near = 0
    for b in range(B):
        n = lead + (rows - lead if nn is None else min(max(nn[b], 0), rows - lead))
        assert (tokens[b, n:] == NOT_DRAWN).all() and (logp[b, n:] == 9.0).all()
        par = {k: (np.float32(v[b]).item() if k != "top_k" else v[b]) for k, v in how.items()}
        for r in range(n):
            row = x[b, r].double().numpy()
            t, lp, gap = lat.draw_row(row, np.float32(u[b, r].item()), **par)
            if gap <= room:
                near += 1
                continue
            assert tokens[b, r] == t, (b, r, tokens[b, r], t, gap, par, float(u[b, r]))
            if t < 0:
                assert logp[b, r] == -np.inf
            else:                                                 # rounded to fp32, of a sum off by `room`
                assert abs(logp[b, r] - lp) <= ref.U32 * abs(lp) + 4 * room + 1e-12, (b, r, logp[b, r], lp)
    assert near <= 1 + B * rows // 50, near


def rows_of_all_kinds(rs, n, V):
    """Peaked, broad, flat, equal, masked, two-valued rows."""
    x = rs.standard_normal((n, V)) * 2
    for i in range(n):
        kind = i % 6
        if kind < 2:
            ids = rs.randint(0, V, 20)
            x[i, ids] += rs.exponential(2.0, 20) + (9 if kind == 0 else 5)
        elif kind == 3:
            x[i] = rs.choice([-1.5, 0.25, 2.0], V)
        elif kind == 4:
            x[i, rs.rand(V) < 0.9] = -np.inf
        elif kind == 5:
            x[i] *= 5
    return torch.from_numpy(x)


HOW = [dict(), dict(top_k=7), dict(top_k=50, top_p=0.95, temperature=0.7), dict(top_p=0.9), dict(min_p=0.05),
       dict(temperature=1.7, top_p=0.995), dict(temperature=0.0), dict(top_k=1), dict(top_p=0.1, temperature=0.3),
       dict(top_k=1000, top_p=0.98, min_p=0.01, temperature=0.8), dict(min_p=1.0), dict(top_p=0.0), dict(top_k=3, min_p=0.5)]
OFF = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def settings(n, first=0):
    rows = [dict(OFF, **HOW[(first + i) % len(HOW)]) for i in range(n)]
    return {k: [r[k] for r in rows] for k in OFF}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 64, 65, 1000, 4097, 32000, 151936])
def test_all_settings_and_sizes(device, dtype, V):
    rs = np.random.RandomState(V)
    B, rows = len(HOW), 6
    if V > 100000:
        rows = 4
    x = rows_of_all_kinds(rs, B * rows, V).view(B, rows, V).to(dtype)
    u = torch.from_numpy(rs.rand(B, rows).astype(np.float32)).clamp(max=1 - 2.0 ** -24)
    u[0, 0], u[-1, -1] = 0.0, 1 - 2.0 ** -24
    how = settings(B)
    say(dtype, V)
    check(x, u, *draw(device, x, u, **how), **how)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("shift", [0.0, 300.0, -300.0])
def test_logits_of_all_magnitudes(device, dtype, shift):
    """Magnitudes from 2^-40 to 2^4, so that cuts fall among tiny logits, too;
    limits of more tokens than a list holds; hot and cold rows."""
    rs = np.random.RandomState(21)
    how = [dict(), dict(top_p=0.3), dict(top_p=0.5), dict(top_p=0.9), dict(top_k=5000), dict(top_k=12000, top_p=0.7),
           dict(top_k=1500, min_p=0.3), dict(top_p=0.8, min_p=0.02), dict(temperature=50.0, top_p=0.6),
           dict(temperature=0.02, top_p=0.9), dict(temperature=1e4), dict(temperature=50.0, min_p=0.999)]
    B, rows, V = len(how), 3, 20011
    x = np.exp2(rs.uniform(-40, 4, (B, rows, V))) * rs.choice([-1, 1], (B, rows, V))
    x[:, 1] = np.exp2(rs.uniform(-40, -20, (B, V))) * rs.choice([-1, 1], (B, V))      # nothing but tiny ones
    x[:, 2, ::2] = 0.0                                            # thousands of ties in the middle
    x = torch.from_numpy(x + shift).to(dtype)
    u = torch.from_numpy(rs.rand(B, rows).astype(np.float32))
    how = {k: [dict(OFF, **h)[k] for h in how] for k in OFF}
    check(x, u, *draw(device, x, u, **how), **how)


@pytest.mark.gpu
def test_trees_and_rows_behind_the_last_node(device):
    rs = np.random.RandomState(1)
    B, rows, V = 5, 9, 777
    x, u = rows_of_all_kinds(rs, B * rows, V).view(B, rows, V).float(), torch.from_numpy(rs.rand(B, rows).astype(np.float32))
    how, nn = settings(B, 2), [7, 0, -3, 30, 2]
    check(x, u, *draw(device, x, u, nn=nn, lead=2, **how), nn=nn, lead=2, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [5, 3000, 40001])
def test_equal_logits_go_by_id(device, V):
    """Sums of equal weights are exact: every border is met exactly."""
    n = 16
    x = torch.zeros(1, n, V)
    u = (torch.arange(n) / n).view(1, n)
    for k, p in ((0, 1.0), (4, 1.0), (0, 0.5), (5, 0.5)):
        tokens, logp = draw(device, x, u, top_k=[k], top_p=[p])
        left = min(k or V, V)
        left = max(1, math.ceil(left * p))
        want = [int(math.floor(i / n * left)) for i in range(n)]
        assert tokens[0].tolist() == want and np.allclose(logp, -math.log(left), rtol=1e-6)
    y = x.clone()
    y[:, :, 0] = -0.0                                             # as large as 0
    assert (draw(device, y, u)[0] == draw(device, x, u)[0]).all()
    assert (draw(device, y, u, top_k=[1])[0] == 0).all()


@pytest.mark.gpu
def test_odd_parameters(device):
    rs = np.random.RandomState(4)
    V, B = 5003, 8
    x = rows_of_all_kinds(rs, B, V).view(B, 1, V).float()
    u = torch.from_numpy(rs.rand(B, 1).astype(np.float32))
    plain = draw(device, x, u)
    for off in (dict(top_k=[0] * B), dict(top_k=[-5] * B), dict(top_k=[V] * B), dict(top_k=[2 ** 31 - 1] * B),
                dict(top_p=[1.0] * B), dict(top_p=[7.0] * B), dict(top_p=[math.nan] * B), dict(min_p=[0.0] * B),
                dict(min_p=[-1.0] * B), dict(min_p=[math.nan] * B), dict(temperature=[1.0] * B)):
        got = draw(device, x, u, **off)
        assert (got[0] == plain[0]).all() and (got[1] == plain[1]).all(), off
    best = x.argmax(-1).numpy()
    for one in (dict(top_k=[1] * B), dict(top_p=[0.0] * B), dict(top_p=[-1.0] * B), dict(min_p=[3.0] * B),
                dict(min_p=[math.inf] * B), dict(temperature=[0.0] * B), dict(temperature=[-1.0] * B),
                dict(temperature=[math.nan] * B), dict(temperature=[1e-30] * B)):
        keep = [b for b in range(B) if b % 6 != 3 or not ({"temperature"} & set(one)) or one["temperature"][0] != 1e-30]
        got = draw(device, x, u, **one)
        assert (got[0][keep] == best[keep]).all() and (got[1][keep] == 0).all(), one
    hot = draw(device, x, u, temperature=[math.inf] * B)          # every finite logit weighs the same
    for b in range(B):
        ids = np.flatnonzero(np.isfinite(x[b, 0].numpy()))
        assert hot[0][b, 0] == ids[int(math.floor(np.float64(np.float32(u[b, 0].item())) * len(ids)))]
    for bad in (1.0, 2.0, -1.0, math.nan, math.inf, -math.inf):   # u outside its range: a token that stays
        got = draw(device, x, torch.full((B, 1), bad))[0]
        ids = [np.flatnonzero(np.isfinite(x[b, 0].numpy())) for b in range(B)]
        assert all(got[b, 0] in ids[b] for b in range(B))
        if bad >= 1:
            assert all(math.exp(float(x[b, 0, got[b, 0]] - x[b, 0].max())) > 0 for b in range(B))


@pytest.mark.gpu
def test_empty_and_unspecified_rows(device):
    V = 1000
    x = torch.full((6, 1, V), -math.inf)
    x[1, 0, 77] = -1e30
    x[2, 0, :] = -3.4e38
    x[3, 0, 5], x[3, 0, 9] = math.nan, 1.0
    x[4, 0, 5], x[4, 0, 9] = math.inf, 1.0
    x[5, 0, :] = math.nan
    u = torch.full((6, 1), 0.5)
    for how in HOW:
        par = {k: [v] * 6 for k, v in dict(OFF, **how).items()}
        tokens, logp = draw(device, x, u, **par)
        assert tokens[0, 0] == -1 and logp[0, 0] == -math.inf
        assert tokens[1, 0] == 77 and logp[1, 0] == 0
        assert 0 <= tokens[2, 0] < V
        assert ((tokens[3:] >= -1) & (tokens[3:] < V)).all()


@pytest.mark.gpu
def test_rows_do_not_depend_on_each_other(device):
    """The same row gives the same token alone, in a batch, and again."""
    rs = np.random.RandomState(6)
    B, rows, V = 40, 3, 30011                                     # (rows at all alignments)
    x = rows_of_all_kinds(rs, B * rows, V).view(B, rows, V).bfloat16()
    u = torch.from_numpy(rs.rand(B, rows).astype(np.float32))
    how = settings(B)
    whole = draw(device, x, u, **how)
    again = draw(device, x, u, **how)
    assert (whole[0] == again[0]).all() and (whole[1] == again[1]).all()
    for b in (0, 2, 3, 9, 17, 39):
        one = draw(device, x[b:b + 1, 1:2].contiguous(), u[b:b + 1, 1:2].contiguous(), **{k: v[b:b + 1] for k, v in how.items()})
        assert one[0][0, 0] == whole[0][b, 1] and one[1][0, 0] == whole[1][b, 1]


@pytest.mark.gpu
def test_frequencies_of_drawn_tokens(device):
    """Evenly spaced u: each token's share is its probability, within one step."""
    V, n = 50, 4000
    rs = np.random.RandomState(9)
    x = torch.from_numpy(rs.standard_normal(V)).float()
    u = ((torch.arange(n) + 0.5) / n).float().view(1, n)
    tokens, _ = draw(device, x.expand(1, n, V).contiguous(), u, top_k=[20])
    w = np.exp(x.double().numpy())
    w[np.argsort(-w)[20:]] = 0
    share = np.bincount(tokens[0], minlength=V) / n
    assert np.abs(share - w / w.sum()).max() <= 1 / n + 1e-6


@pytest.mark.gpu
def test_two_streams_and_a_captured_call(device):
    rs = np.random.RandomState(12)
    B, rows, V = 6, 2, 20000
    xs = [rows_of_all_kinds(rs, B * rows, V).view(B, rows, V).float() for _ in range(3)]
    us = [torch.from_numpy(rs.rand(B, rows).astype(np.float32)) for _ in range(3)]
    how = settings(B, 2)
    want = [draw(device, x, u, **how) for x, u in zip(xs, us)]
    kinds = dict(temperature=F32, top_k=I32, top_p=F32, min_p=F32)
    par = {k: torch.tensor(v, dtype=kinds[k], device=device) for k, v in how.items()}
    need = max(bd.dt_sample_workspace(xs[0].to(device)), 16)
    side = []
    for x, u in zip(xs, us):
        side.append((torch.cuda.Stream(), x.to(device), u.to(device), torch.zeros(B, rows, dtype=I32, device=device),
                     torch.empty(need, dtype=torch.uint8, device=device)))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, u, t, ws in side:
            bd.dt_sample_rows(x, u, t, workspace=ws, stream=s, **par)
    torch.cuda.synchronize()
    for (_, _, _, t, _), w in zip(side, want):
        assert (t.cpu().numpy() == w[0]).all()
    x, u = torch.zeros_like(side[0][1]), torch.zeros_like(side[0][2])
    t, lp, ws = torch.zeros(B, rows, dtype=I32, device=device), torch.zeros(B, rows, device=device), side[0][4]
    bd.dt_sample_rows(x, u, t, logp=lp, workspace=ws, **par)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.dt_sample_rows(x, u, t, logp=lp, workspace=ws, **par)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        u.copy_(us[i])
        graph.replay()
        torch.cuda.synchronize()
        assert (t.cpu().numpy() == want[i][0]).all() and (lp.cpu().numpy() == want[i][1]).all()


@pytest.mark.gpu
def test_logits_behind_32_bits(device):
    """Rows that begin behind 2^31 elements."""
    V, rows = (1 << 25) + 3, 66
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("no room")
    x = torch.zeros(1, rows, V, dtype=BF16, device=device)
    x[0, rows - 1, V - 2], x[0, 1, 12345] = 20.0, 30.0
    u = torch.full((1, rows), 0.25, device=device)
    tokens = torch.zeros(1, rows, dtype=I32, device=device)
    need = bd.dt_sample_workspace(x)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    for how, mid in ((dict(), V // 4), (dict(min_p=[0.5]), V // 4), (dict(top_k=[1 << 20]), 1 << 18)):
        par = {k: torch.tensor(v, dtype=I32 if k == "top_k" else F32, device=device) for k, v in how.items()}
        bd.dt_sample_rows(x, u, tokens, workspace=ws, **par)
        torch.cuda.synchronize()
        got = tokens.cpu()[0]
        assert int(got[1]) == 12345 and int(got[2]) == mid and int(got[rows - 2]) == mid
        assert int(got[rows - 1]) == V - 2


@pytest.mark.gpu
def test_counts_of_nodes_at_the_ends_of_their_type(device):
    rs = np.random.RandomState(31)
    nn = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 3, -1, 8]
    B, rows, V = len(nn), 9, 333
    x, u = rows_of_all_kinds(rs, B * rows, V).view(B, rows, V).float(), torch.from_numpy(rs.rand(B, rows).astype(np.float32))
    for lead in (1, 2, 9):
        check(x, u, *draw(device, x, u, nn=nn, lead=lead), nn=nn, lead=lead)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [128, 131, 256])
def test_calls_of_so_many_rows_that_their_threads_pass_32_bits(device, B):
    """2^23 rows and more, up to the documented 2^24: tokens of two logits."""
    rows, lead = 65536, 3
    g = torch.Generator(device=device).manual_seed(B)
    x = torch.randn(B, rows, 2, generator=g, device=device)
    u = torch.rand(B, rows, generator=g, device=device)
    nn = torch.randint(0, rows - lead + 1, (B,), generator=g, device=device, dtype=I32)
    nn[-1] = rows - lead
    tokens = torch.full((B, rows), NOT_DRAWN, dtype=I32, device=device)
    bd.dt_sample_rows(x, u, tokens, lead=lead, n_nodes=nn)
    torch.cuda.synchronize()
    first = 1 / (1 + torch.exp(x[..., 1].double() - x[..., 0].double()))      # the first one's share
    drawn = torch.arange(rows, device=device)[None] < lead + nn[:, None]
    near = drawn & ((first - u.double()).abs() < 1e-12)           # (weights are off by 2^-43, shares by little more)
    assert int(near.sum()) < 10
    want = torch.where(drawn, (u.double() >= first).int(), NOT_DRAWN)
    assert ((tokens == want) | near).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
def test_nan_counts_as_minus_infinity(device, dtype):
    """Rows masked with NaN of all kinds, whole 16-byte groups of them among
    them, give the tokens of rows masked with -inf."""
    rs = np.random.RandomState(33)
    V, rows = 32000, 12
    how = HOW + [dict(top_k=600), dict(top_k=900, top_p=0.99), dict(top_p=0.999, temperature=3.0), dict(top_k=5000)]
    B = len(how)
    x = torch.from_numpy(rs.standard_normal((B, rows, V))).to(dtype)
    gone = torch.from_numpy(np.repeat(rs.rand(B, rows, V // 16) < 0.9, 16, -1) | (rs.rand(B, rows, V) < 0.05))
    # an exponent of ones, any fraction but 0 and any sign: quiet and signalling ones
    fraction, ints = (7, np.int16) if dtype == BF16 else (23, np.int32)
    bits = (255 << fraction) + rs.randint(1, 1 << fraction, x.shape) - (rs.randint(0, 2, x.shape) << (fraction + 8))
    nan = torch.from_numpy(bits.astype(ints)).view(dtype)
    assert torch.isnan(nan).all() and (nan.view(torch.int16 if dtype == BF16 else I32) < 0).any()
    u = torch.from_numpy(rs.rand(B, rows).astype(np.float32))
    how = {k: [dict(OFF, **h)[k] for h in how] for k in OFF}
    want = draw(device, x.masked_fill(gone, -math.inf), u, **how)
    got = draw(device, torch.where(gone, nan, x), u, **how)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
    assert draw(device, nan, u, **how)[0].max() == -1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("temperature", [1.0, 1e-30, 1e-36])
def test_zeros_of_both_signs_are_one_value(device, dtype, temperature):
    """They tie by id, also where the temperature is so low that nothing but
    zeros weighs anything."""
    rs = np.random.RandomState(34)
    V, rows = 6000, 16
    how = [dict(top_p=0.6), dict(top_p=0.3), dict(top_k=1700), dict(top_k=1700, top_p=0.7), dict(top_k=1700, min_p=0.5),
           dict(top_k=5), dict(min_p=0.5), dict(top_p=0.95)]
    B = len(how)
    x = torch.from_numpy(np.where(rs.rand(B, rows, V) < 0.5, 0.0, -1.0)).to(dtype)
    signed = torch.where((x == 0) & torch.from_numpy(rs.rand(B, rows, V) < 0.5), -0.0, x.float()).to(dtype)
    u = ((torch.arange(rows) + 0.5) / rows).expand(B, rows).contiguous()
    how = dict({k: [dict(OFF, **h)[k] for h in how] for k in OFF}, temperature=[temperature] * B)
    want = draw(device, x, u, **how)
    got = draw(device, signed, u, **how)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
    check(signed, u, *got, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("temperature", [1.0, 1e4, 1e8, 1e15, 1e30, 3e38, math.inf])
def test_min_p_goes_by_the_rounded_weights(device, dtype, temperature):
    """Whichever way a row goes: a top_p that leaves everything with any weight
    in its row (6000 alike are each above 2^-24 of the sum) takes another way than
    min_p alone."""
    rs = np.random.RandomState(35)
    least = [1.0, 1 - 2.0 ** -24, 1 - 2.0 ** -22, 0.999, 0.5, 2.5]
    B, rows, V = len(least), 8, 6000
    x = rs.standard_normal((B, rows, V))
    x[:, ::2] = np.maximum(x[:, ::2], 1.0)                        # (thousands of tokens, and rows with few of them)
    x[:, 1, rs.rand(V) < 0.1] = -np.inf
    x = torch.from_numpy(x).to(dtype)
    u = ((torch.arange(rows) + 0.5) / rows).expand(B, rows).contiguous()
    how = dict(temperature=[temperature] * B, min_p=least)
    got = draw(device, x, u, **how)
    want = draw(device, x, u, top_p=[1 - 2.0 ** -24] * B, **how)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()
    if temperature >= 1e30:                                       # all weights are 1
        for b in range(B - 1):                                    # (and the last one asks for more)
            for r in range(rows):
                ids = np.flatnonzero(np.isfinite(x[b, r].float().numpy()))
                assert got[0][b, r] == ids[int((r + 0.5) / rows * len(ids))]
