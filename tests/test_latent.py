"""Latent attention (dt_latent_append, dt_latent_attention, dt_latent_prefill,
dt_latent_commit) against its definitions in 64 bits (latent_ref.py)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import latent_ref as lat
import pass_ref as ref

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
BAD, LIMIT, WORK = bd.DT_ERR_INVALID_ARG, bd.DT_ERR_UNSUPPORTED, bd.DT_ERR_WORKSPACE
SENTINEL = 7.0
FAKE = 0x100000


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# refusals (no GPU)
# ---------------------------------------------------------------------------

def _struct(cls, base, kw):
    s = cls()
    for k, v in dict(base, **kw).items():
        setattr(s, k, v)
    return s


def _cache(**kw):
    return _struct(bd._LatentCache, dict(c=FAKE, page_table=FAKE, layer_stride=1 << 20, page_stride=16384,
                                         slot_stride=576, layers=2, num_pages=9, page_size=16, max_pages=8, Dc=512,
                                         Dr=64, dtype=bd.DT_DTYPE_BF16), kw)


def _chunk(**kw):
    return _struct(bd._Chunk, dict(B=2, lead=1, n_max=8, ctx_len=FAKE), kw)


def _append(**kw):
    return _struct(bd._LatentAppendParams,
                   dict(latent=FAKE, k_rot=FAKE, q_rot=FAKE, q_out=2 * FAKE, latent_stride=576, k_stride=576,
                        q_stride=4096, q_head_stride=192, q_out_stride=9216, q_out_head_stride=576, Hq=16, eps=1e-6,
                        freqs=FAKE, rot_scale=1.0), kw)


def _attn(**kw):
    return _struct(bd._LatentParams, dict(q=FAKE, out=2 * FAKE, weight=FAKE, q_stride=9216, out_stride=8192, Hq=16,
                                          Dn=128, max_keys=100, scale=0.1, workspace=FAKE, workspace_bytes=1 << 40), kw)


def _commit(**kw):
    return _struct(bd._CommitParams, dict(tokens=FAKE, parents=FAKE, target=FAKE, L=9, accepted=FAKE, lengths=FAKE), kw)


CALLS = {"dt_latent_append": _append, "dt_latent_attention": _attn, "dt_latent_prefill": _attn,
         "dt_latent_commit": _commit}


def call(name, cache, chunk, p):
    return getattr(bd._load(), name)(*(ctypes.byref(x) if x is not None else None for x in (cache, chunk, p)))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(c=None), BAD), (dict(c=FAKE + 8), BAD), (dict(page_table=None), BAD), (dict(page_table=FAKE + 2), BAD),
    (dict(layers=0), BAD), (dict(num_pages=0), BAD), (dict(page_size=0), BAD), (dict(max_pages=0), BAD),
    (dict(Dc=0), BAD), (dict(Dr=0), BAD), (dict(dtype=0), BAD), (dict(dtype=3), BAD), (dict(layer_stride=4), BAD),
    (dict(page_stride=-8), BAD), (dict(slot_stride=577), BAD), (dict(Dc=128), LIMIT), (dict(Dc=513), LIMIT),
    (dict(Dr=16), LIMIT), (dict(Dr=128), LIMIT), (dict(page_size=1 << 16, max_pages=1 << 15), LIMIT),
])
def test_bad_caches_are_refused(name, kw, status):
    assert call(name, _cache(**kw), _chunk(), CALLS[name]()) == status


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(lead=-1), BAD), (dict(n_max=-1), BAD), (dict(lead=0, n_max=0), BAD),
    (dict(ctx_len=None), BAD), (dict(ctx_len=FAKE + 1), BAD), (dict(n_nodes=FAKE + 2), BAD), (dict(mask=FAKE + 1), BAD),
    (dict(B=65536), LIMIT), (dict(lead=65530), LIMIT), (dict(B=4096, n_max=4096), LIMIT),
])
def test_bad_chunks_are_refused(name, kw, status):
    assert call(name, _cache(), _chunk(**kw), CALLS[name]()) == status


@pytest.mark.parametrize("axis", ["layer_stride", "page_stride", "slot_stride"])
def test_writes_into_overlapping_tokens_are_refused(axis):
    for name in ("dt_latent_append", "dt_latent_commit"):
        assert call(name, _cache(**{axis: 568}), _chunk(), CALLS[name]()) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(latent=None), BAD), (dict(k_rot=None), BAD), (dict(q_out=None), BAD), (dict(q_rot=None), BAD),
    (dict(latent=FAKE + 2), BAD), (dict(k_rot=FAKE + 8), BAD), (dict(q_out=FAKE + 4), BAD), (dict(norm=FAKE + 8), BAD),
    (dict(freqs=FAKE + 4), BAD), (dict(latent_stride=504), BAD), (dict(latent_stride=513), BAD), (dict(k_stride=56), BAD),
    (dict(q_stride=2936), BAD), (dict(q_head_stride=56), BAD), (dict(q_head_stride=65), BAD),
    (dict(q_out_head_stride=-576), BAD), (dict(q_head_stride=1 << 62), BAD), (dict(Hq=0), BAD), (dict(Hq=4097), LIMIT),
    (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD), (dict(rot_scale=math.inf), BAD), (dict(layer=2), BAD),
    (dict(layer=-1), BAD), (dict(q_out=FAKE), BAD), (dict(q_out=FAKE, q_out_stride=4096), BAD),
])
def test_append_refusals(kw, status):
    assert call("dt_latent_append", _cache(), _chunk(), _append(**kw)) == status


@pytest.mark.parametrize("name", ["dt_latent_attention", "dt_latent_prefill"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(q=FAKE + 2), BAD), (dict(out=2 * FAKE + 8), BAD),
    (dict(out=FAKE), BAD), (dict(q_stride=2000), BAD), (dict(q_stride=9220), BAD), (dict(out_stride=2040), BAD),
    (dict(Hq=0), BAD), (dict(Hq=4097), LIMIT), (dict(scale=0.0), BAD), (dict(scale=math.nan), BAD),
    (dict(scale=math.inf), BAD), (dict(lse=FAKE + 2), BAD), (dict(layer=2), BAD), (dict(layer=-1), BAD),
    (dict(workspace=None), WORK), (dict(workspace=FAKE + 8), WORK), (dict(workspace_bytes=100), WORK),
])
def test_attention_refusals(name, kw, status):
    assert call(name, _cache(), _chunk(), _attn(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(weight=None), BAD), (dict(weight=FAKE + 8), BAD), (dict(Dn=0), BAD), (dict(max_keys=0), BAD),
    (dict(Dn=96), LIMIT), (dict(Dn=256), LIMIT),
])
def test_prefill_refusals(kw, status):
    assert call("dt_latent_prefill", _cache(), _chunk(), _attn(**kw)) == status


def test_workspaces_and_limits_of_a_call():
    lib, big = bd._load(), _chunk(B=1, lead=0, n_max=65536)
    assert lib.dt_latent_workspace(ctypes.byref(_cache()), ctypes.byref(_chunk()), 16) > 0
    assert lib.dt_latent_workspace(ctypes.byref(_cache(Dc=100)), ctypes.byref(_chunk()), 16) == 0
    assert lib.dt_latent_workspace(ctypes.byref(_cache()), ctypes.byref(_chunk(B=2000, lead=0, n_max=2000)), 4096) == 0
    assert lib.dt_latent_prefill_workspace(ctypes.byref(_cache()), ctypes.byref(big), 16, 96, 100) == 0
    assert lib.dt_latent_prefill_workspace(ctypes.byref(_cache()), ctypes.byref(big), 16, 64, 0) == 0
    a = lib.dt_latent_prefill_workspace(ctypes.byref(_cache()), ctypes.byref(_chunk()), 16, 128, 1000)
    b = lib.dt_latent_prefill_workspace(ctypes.byref(_cache()), ctypes.byref(_chunk()), 16, 128, 2000)
    assert abs((b - a) - 2 * 16 * 1000 * 512) <= 256
    # 2^30 slots of 4096 heads of 65535 requests: bytes that 64 bits hold
    c = _chunk(B=65535)
    assert lib.dt_latent_prefill_workspace(ctypes.byref(_cache()), ctypes.byref(c), 3000, 128, 1 << 30) > 1 << 56


def test_prefill_workspaces_that_no_buffer_can_have():
    """The made keys' and values' bytes are counted exactly, and a product that
    passes 63 bits neither wraps to a small size nor lets a call through."""
    lib, one = bd._load(), _chunk(B=65535, lead=1, n_max=0)

    def size(chunk, Hq, Dn, keys):
        return lib.dt_latent_prefill_workspace(ctypes.byref(_cache()), ctypes.byref(chunk), Hq, Dn, keys)
    for keys in (1 << 20, (1 << 30) - 1):
        assert size(one, 100, 64, keys) - size(one, 100, 64, 1) == 65535 * 100 * 4 * 64 * (keys - 1)
    # bytes 2^63 - 2^49 (which fit), 2^63, 2^64, 2^64, and some that would wrap to a middling size
    fits = _chunk(B=16383, lead=1, n_max=0)
    assert size(fits, 1024, 128, 1 << 30) - size(fits, 1024, 128, 1) == 16383 * 1024 * 512 * ((1 << 30) - 1)
    for B, Hq, Dn, keys in ((16384, 1024, 128, 1 << 30), (8192, 4096, 128, 1 << 30), (16384, 4096, 64, 1 << 30),
                            (65535, 3000, 128, 1 << 30), (65535, 4096, 128, 2 ** 31 - 1)):
        chunk = _chunk(B=B, lead=1, n_max=0)
        assert size(chunk, Hq, Dn, keys) == 2 ** 64 - 1
        for room in (1 << 40, 2 ** 64 - 1):
            p = _attn(Hq=Hq, Dn=Dn, max_keys=keys, q_stride=Hq * (Dn + 64), out_stride=Hq * Dn, workspace_bytes=room)
            assert call("dt_latent_prefill", _cache(), chunk, p) == LIMIT


def test_empty_batches_and_null_structs():
    cache, none, full = _cache(c=None, page_table=None), _chunk(B=0, ctx_len=None), _chunk()
    assert call("dt_latent_append", cache, none, _append(latent=None)) == bd.DT_OK
    assert call("dt_latent_attention", cache, none, _attn(q=None, workspace=None)) == bd.DT_OK
    assert call("dt_latent_prefill", cache, none, _attn(q=None, weight=None, workspace=None)) == bd.DT_OK
    assert call("dt_latent_commit", cache, none, _commit(target=None)) == bd.DT_OK
    for name, p in CALLS.items():
        assert call(name, None, full, p()) == BAD
        assert call(name, _cache(), None, p()) == BAD
        assert call(name, _cache(), full, None) == BAD


def test_binding_checks_tensors():
    c, table = torch.zeros(4, 16, 320, dtype=BF16), torch.zeros(2, 2, dtype=I32)
    cache = bd.LatentCache(c, table, 64)
    assert (cache.Dc, cache.Dr, cache.layers) == (256, 64, 1)
    for bad in (dict(c=c.float()), dict(c=c[..., ::2]), dict(c=c[0]), dict(page_table=table.long()), dict(Dr=0),
                dict(Dr=320), dict(page_table=table[0])):
        with pytest.raises(bd.DtError):
            bd.LatentCache(**dict(dict(c=c, page_table=table, Dr=64), **bad))
    chunk = bd.Chunk(torch.zeros(2, dtype=I32), lead=3)
    q, out = torch.zeros(2, 3, 4, 320, dtype=BF16), torch.zeros(2, 3, 4, 256, dtype=BF16)
    for bad in (dict(q=q.half()), dict(q=q[:, :2]), dict(q=q[..., :256]), dict(out=q), dict(q=q[0]),
                dict(lse=torch.zeros(2, 3, 3)), dict(q=torch.zeros(2, 3, 8, 320, dtype=BF16)[:, :, ::2])):
        with pytest.raises(bd.DtError):
            bd.dt_latent_attention(cache, chunk, **dict(dict(q=q, out=out, scale=0.1), **bad))
    q, out, w = torch.zeros(2, 3, 4, 192, dtype=BF16), torch.zeros(2, 3, 4, 128, dtype=BF16), torch.zeros(4, 256, 256, dtype=BF16)
    for bad in (dict(weight=w[:3]), dict(weight=w.half()), dict(q=q[..., :128]), dict(out=out[..., :64]),
                dict(weight=w.transpose(1, 2))):
        with pytest.raises(bd.DtError):
            bd.dt_latent_prefill(cache, chunk, **dict(dict(q=q, weight=w, out=out, scale=0.1, max_keys=32), **bad))
    x, k = torch.zeros(2, 3, 256, dtype=BF16), torch.zeros(2, 3, 64, dtype=BF16)
    qr = torch.zeros(2, 3, 4, 64, dtype=BF16)
    for bad in (dict(latent=x[..., :64]), dict(k_rot=x), dict(norm=torch.zeros(64, dtype=BF16)), dict(latent=x[0]),
                dict(freqs=torch.zeros(32)), dict(freqs=torch.zeros(64, dtype=torch.float64)), dict(q_rot=qr[..., :32]),
                dict(q_rot=qr, q_out=qr[:, :, :2]), dict(q_rot=qr)):
        with pytest.raises(bd.DtError):
            bd.dt_latent_append(cache, chunk, **dict(dict(latent=x, k_rot=k), **bad))
    for fn in (lambda: bd.dt_latent_append(cache, chunk, x, k),
               lambda: bd.dt_latent_attention(cache, chunk, torch.zeros(2, 3, 4, 320, dtype=BF16),
                                              torch.zeros(2, 3, 4, 256, dtype=BF16), 0.1),
               lambda: bd.dt_latent_prefill(cache, chunk, q, w, out, 0.1, 32),
               lambda: bd.dt_latent_commit(cache, chunk, None, None, torch.zeros(2, 3, dtype=I32),
                                           torch.zeros(2, 4, dtype=I32), torch.zeros(2, dtype=I32))):
        with pytest.raises(bd.DtError, match="must be on a GPU"):           # host tensors are out of kernels' reach
            fn()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def upload(t, device):
    return None if t is None else (torch.from_numpy(t) if isinstance(t, np.ndarray) else t).to(device)


def chunk_on(device, ctx, lead, n_max, nn, seen=None, depths=None):
    return bd.Chunk(torch.tensor(ctx, dtype=I32, device=device), lead, n_max,
                    None if nn is None else torch.tensor(nn, dtype=I32, device=device),
                    None if seen is None else upload(ref.pack_bits(seen), device), upload(depths, device))


def test_every_call_goes_through_its_device(monkeypatch):
    """The entry points that launch are called by way of their tensors' device."""
    seen = []
    monkeypatch.setattr(bd, "_on_device", lambda index, call, *args: seen.append((index, call.__name__)) or 0)
    cache = bd.LatentCache(torch.zeros(2, 16, 288, dtype=BF16), torch.zeros(1, 2, dtype=torch.int32), 32)
    chunk = bd.Chunk(torch.zeros(1, dtype=torch.int32))
    x, q = torch.zeros(1, 1, 288, dtype=BF16), torch.zeros(1, 1, 2, 288, dtype=BF16)
    i32 = torch.zeros(1, 1, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    bd.dt_latent_append(cache, chunk, x[..., :256], x[..., 256:])
    bd.dt_latent_attention(cache, chunk, q, torch.empty(1, 1, 2, 256, dtype=BF16), 1.0, workspace=ws)
    bd.dt_latent_prefill(cache, chunk, q[..., :96].contiguous(), torch.zeros(2, 128, 256, dtype=BF16),
                         torch.empty(1, 1, 2, 64, dtype=BF16), 1.0, 32, workspace=ws)
    bd.dt_latent_commit(cache, chunk, None, None, i32, i32.clone(), torch.zeros(1, dtype=torch.int32))
    bd.dt_sample_rows(torch.zeros(1, 1, 32), torch.zeros(1, 1), i32)
    assert seen == [(-1, name) for name in ("dt_latent_append", "dt_latent_attention", "dt_latent_prefill",
                                            "dt_latent_commit", "dt_sample_rows")]


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    dict(dtype=BF16, Dc=512, Dr=64, Hq=16, lead=1, n_max=0, nn=None, ctx=[4000], P=16),
    dict(dtype=F16, Dc=256, Dr=32, Hq=5, lead=2, n_max=9, nn=[9, 0, 4, 30, 3], ctx=[0, 7, 100000, 33, -1], P=24, tree=True),
    dict(dtype=BF16, Dc=256, Dr=64, Hq=33, lead=0, n_max=50, nn=[50, 1], ctx=[3, 61], P=1, interleaved=True),
    dict(dtype=F16, Dc=512, Dr=32, Hq=128, lead=0, n_max=17, nn=[17, 16], ctx=[5, 1 << 20], P=64, norm=False, scale=1.25),
    dict(dtype=BF16, Dc=512, Dr=64, Hq=0, lead=1, n_max=3, nn=[3, 2, 1], ctx=[9, 2, 0], P=16, tree=True),
    dict(dtype=BF16, Dc=512, Dr=64, Hq=3, lead=1, n_max=3, nn=[3, 2], ctx=[9, 2], P=16, turn=False, norm=False),
    dict(dtype=F16, Dc=256, Dr=64, Hq=1, lead=3, n_max=700, nn=[700, 651, 2], ctx=[1, 2, 3], P=8, interleaved=True),
], ids=str)
def test_append(device, case):
    say(case)
    rs = np.random.RandomState(len(str(case)))
    dtype, Dc, Dr, Hq, lead, n_max, P = (case[k] for k in ("dtype", "Dc", "Dr", "Hq", "lead", "n_max", "P"))
    ctx, nn, B, rows, eps = case["ctx"], case["nn"], len(case["ctx"]), lead + n_max, 1e-5
    far = max(ctx) > 5000
    depths = seen = None
    if case.get("tree"):
        _, depths, seen = ref.random_tree(rs, B, n_max, [min(n, n_max) for n in nn])
    c, table = lat.make_latents(rs, [min(x, 300) for x in ctx] if far else ctx, rows, P, Dc + Dr, dtype, layers=2,
                                width=(max(ctx) + rows) // P + 1)
    if far:                                                       # far slots on the few pages there are
        for b, n in enumerate(ctx):
            have = table[b][table[b] >= 0]
            if n > 300:
                table[b, n // P:(n + rows) // P + 1] = have[:(n + rows) // P + 1 - n // P]
    down = torch.from_numpy(rs.standard_normal((B, rows, Dc + Dr + 8))).to(dtype)
    q = torch.from_numpy(rs.standard_normal((B, rows, max(Hq, 1), 128 + Dr))).to(dtype)
    norm = torch.from_numpy(1 + 0.2 * rs.standard_normal(Dc)).to(dtype) if case.get("norm", True) else None
    freqs = 10000.0 ** (-np.arange(0, Dr, 2) / Dr) if case.get("turn", True) else None
    scale = case.get("scale", 1.0)
    dc, ddown, dq = c.clone().to(device), down.to(device), q.to(device)
    out = torch.full((B, rows, max(Hq, 1), Dc + Dr), SENTINEL, dtype=dtype, device=device)
    bd.dt_latent_append(bd.LatentCache(dc, upload(table, device), Dr), chunk_on(device, ctx, lead, n_max, nn, seen, depths),
                        ddown[..., :Dc], ddown[..., Dc:Dc + Dr], q_rot=dq[..., 128:] if Hq else None,
                        q_out=out[..., Dc:] if Hq else None, norm=upload(norm, device), eps=eps, freqs=upload(freqs, device),
                        interleaved=case.get("interleaved", False), rot_scale=scale, layer=1)
    torch.cuda.synchronize()
    want, touched = c.clone(), torch.zeros(c.shape[:3], dtype=torch.bool)
    got, out = dc.cpu(), out.cpu()
    for b in range(B):
        for r in range(rows):
            if r >= ref.rows_of(b, ctx, lead, n_max, nn):
                assert (out[b, r] == SENTINEL).all()
                continue
            pos = ctx[b] + r if depths is None or r < lead else ctx[b] + lead - 1 + depths[b, r - lead]
            fr, il = freqs, case.get("interleaved", False)

            def check(x, row, w):
                if fr is None and w is None:
                    assert torch.equal(x, row)
                    return
                y, size = ref.append_head(row.double().numpy(), None if w is None else w.double().numpy(), eps, pos,
                                          fr if w is None else None, il, scale)
                tol = ref.append_tolerance(y, size, dtype)
                if w is not None:                                 # up to 512 squares: 8 in a lane, then a tree of six
                    tol = tol + 16 * ref.U32 * size
                assert (np.abs(x.double().numpy() - y) <= tol).all()

            at = ref.slot_at(table, c.shape[1], P, b, ctx[b] + r)
            if at is not None:
                x = got[1, at[0], at[1]]
                if norm is None:
                    assert torch.equal(x[:Dc], down[b, r, :Dc])
                else:
                    check(x[:Dc], down[b, r, :Dc], norm)
                check(x[Dc:], down[b, r, Dc:Dc + Dr], None)
                touched[1, at[0], at[1]] = True
            for h in range(Hq):
                check(out[b, r, h, Dc:], q[b, r, h, 128:], None)
    assert (out[..., :Dc] == SENTINEL).all()
    keep = ~touched
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))


@pytest.mark.gpu
def test_append_in_place_and_bad_pages(device):
    rs = np.random.RandomState(3)
    c, table = lat.make_latents(rs, [10, 10, 20], 4, 8, 576, BF16)
    table[0, 1], table[1, 1] = -5, c.shape[1]                     # slots 8.. of these have no page
    before = c.clone()
    q = torch.from_numpy(rs.standard_normal((3, 4, 6, 64))).to(BF16)
    x = torch.from_numpy(rs.standard_normal((3, 4, 576))).to(BF16).to(device)
    dc, dq = c.to(device), q.to(device)
    freqs = torch.from_numpy(10000.0 ** (-np.arange(0, 64, 2) / 64))
    bd.dt_latent_append(bd.LatentCache(dc, upload(table, device), 64), chunk_on(device, [10, 10, 20], 4, 0, None),
                        x[..., :512], x[..., 512:], q_rot=dq, q_out=dq, freqs=freqs.to(device))
    other = torch.empty_like(dq)
    bd.dt_latent_append(bd.LatentCache(dc, upload(table, device), 64), chunk_on(device, [10, 10, 20], 4, 0, None),
                        x[..., :512], x[..., 512:], q_rot=q.to(device), q_out=other, freqs=freqs.to(device))
    torch.cuda.synchronize()
    assert torch.equal(dq, other)
    got, mine = dc.cpu(), torch.zeros(c.shape[:3], dtype=torch.bool)
    for r in range(4):
        mine[0, table[2, (20 + r) // 8], (20 + r) % 8] = True
    assert torch.equal(got[~mine].view(torch.int16), before[~mine].view(torch.int16))
    assert torch.equal(got[mine][:, :512], x[2, :, :512].cpu()[torch.argsort(torch.tensor(
        [int(table[2, (20 + r) // 8]) * 8 + (20 + r) % 8 for r in range(4)]))])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def problem(case):
    rs = np.random.RandomState(case.get("seed", 0) + 17 * len(str(case)))
    dtype, Dc, Dr, Hq, lead, n_max, P = (case[k] for k in ("dtype", "Dc", "Dr", "Hq", "lead", "n_max", "P"))
    ctx, nn = case["ctx"], case.get("nn")
    B, rows = len(ctx), lead + n_max
    seen = None
    if case.get("tree"):
        _, _, seen = ref.random_tree(rs, B, n_max, [n_max if nn is None else min(max(n, 0), n_max) for n in nn or [0] * B])
        if case["tree"] == "odd":                                 # any bits at all, rows without one among them
            seen = rs.rand(B, n_max, n_max) < 0.3
            seen[:, ::3] = False
    c, table = lat.make_latents(rs, ctx, rows, P, Dc + Dr, dtype, layers=case.get("layers", 1), sd=case.get("sd", 1.0))
    lat.fill_chunk(rs, c, table, ctx, rows, case.get("sd", 1.0))
    Dn = case.get("Dn")
    q = torch.from_numpy(rs.standard_normal((B, rows, Hq, (Dn or Dc) + Dr))).to(dtype)
    w = None if Dn is None else torch.from_numpy(rs.standard_normal((Hq, 2 * Dn, Dc)) * Dc ** -0.5).to(dtype)
    scale = case.get("scale", (Dn or Dc + Dr) ** -0.5)
    return rs, c, table, q, w, seen, scale


def run_attention(device, case, c, table, q, w, seen, scale, stream=None, max_keys=None):
    lead, n_max, ctx, nn, Hq, Dn = case["lead"], case["n_max"], case["ctx"], case.get("nn"), case["Hq"], case.get("Dn")
    cache = bd.LatentCache(c.to(device), upload(table, device), case["Dr"])
    chunk = chunk_on(device, ctx, lead, n_max, nn, seen)
    dq = q.to(device)
    out = torch.full(tuple(q.shape[:3]) + (Dn or case["Dc"],), SENTINEL, dtype=q.dtype, device=device)
    lse = torch.full(tuple(q.shape[:3]), SENTINEL, dtype=torch.float32, device=device)
    layer = case.get("layers", 1) - 1
    if Dn is None:
        ws = torch.full((bd.dt_latent_workspace(cache, chunk, Hq),), 255, dtype=torch.uint8, device=device)
        bd.dt_latent_attention(cache, chunk, dq, out, scale, lse=lse, layer=layer, workspace=ws, stream=stream)
    else:
        keys = max_keys or max(max(ctx) + lead + n_max, 1)
        ws = torch.full((bd.dt_latent_prefill_workspace(cache, chunk, Hq, Dn, keys),), 255, dtype=torch.uint8, device=device)
        bd.dt_latent_prefill(cache, chunk, dq, w.to(device), out, scale, keys, lse=lse, layer=layer, workspace=ws,
                             stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check_attention(case, c, table, q, w, seen, scale, out, lse, max_keys=None):
    lead, n_max, ctx, nn, Hq, Dc, Dn, P = (case.get(k) for k in ("lead", "n_max", "ctx", "nn", "Hq", "Dc", "Dn", "P"))
    dtype, half = case["dtype"], ref.HALF_STEP[case["dtype"]]
    layer, worst = case.get("layers", 1) - 1, 0.0
    cap = min(table.shape[1] * P, max_keys or 1 << 30)
    every = case.get("every", 1)
    for b in range(len(ctx)):
        n = ref.rows_of(b, ctx, lead, n_max, nn)
        assert (out[b, n:] == SENTINEL).all() and (lse[b, n:] == SENTINEL).all()
        for r in list(range(0, n, every)) + ([n - 1] if n else []):
            row = seen[b, r - lead] if seen is not None and r >= lead else None
            slots = lat.seen_slots(table, c.shape[1], P, b, ctx[b], lead, r, n - lead, row, cap)
            where = [ref.slot_at(table, c.shape[1], P, b, s) for s in slots]
            x = np.stack([c[layer, p, o].double().numpy() for p, o in where]) if where else np.zeros((0, c.shape[-1]))
            qq = q[b, r].double().numpy()
            if Dn is None:
                want, wl, tol, slack = lat.attend(qq, x, x[:, :Dc], scale, dtype)
            else:
                ww = w.double().numpy()
                kv = np.einsum("hnc,sc->hsn", ww, x[:, :Dc])
                # made keys and values: fp32 sums of Dc products, then half a step
                err = ref.U32 * (Dc + 2) * np.einsum("hnc,sc->hsn", np.abs(ww), np.abs(x[:, :Dc])) + half * np.abs(kv) + \
                    ref.SMALLEST[dtype]
                K = np.concatenate((kv[..., :Dn], np.broadcast_to(x[:, Dc:], (Hq,) + x[:, Dc:].shape)), -1)
                move = scale * np.einsum("hd,hsd->hs", np.abs(qq[:, :Dn]), err[..., :Dn]) if where else np.zeros((Hq, 1))
                V = kv[..., Dn:]
                want, wl, tol, slack = lat.attend(qq, K, V, scale, dtype, score_error=move.max(1))
                if where:
                    p = np.exp(scale * np.einsum("hd,hsd->hs", qq, K) - wl[:, None])
                    tol = tol + np.einsum("hs,hsn->hn", p, err[..., Dn:]) * (1 + 4 * half)
            got = out[b, r].double().numpy()
            bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want))    # (a NaN that is seen stays one)
            worst = max(worst, float(np.nanmax(np.append(np.abs(got - want) / tol, 0))))
            assert not bad.any(), (b, r, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], tol[bad][:4])
            gl = lse[b, r].double().numpy()
            if not where:
                assert (gl == -np.inf).all()
            else:
                lt = slack + ref.U32 * (len(slots) + 64 + 4 * np.abs(wl))
                assert ((np.abs(gl - wl) <= lt) | (np.isnan(gl) & np.isnan(wl))).all(), (b, r, gl, wl)
    say("worst error over its bound", round(worst, 3))


SHAPES = [
    dict(lead=1, n_max=0, ctx=[0, 1, 31, 32, 63, 64, 65, 300, -1], P=16),                  # single tokens
    dict(lead=1, n_max=0, ctx=[5000, 17], P=64),                                           # a long one, split
    dict(lead=1, n_max=9, nn=[9, 0, 4, 30, -3], ctx=[0, 7, 130, 33, 20], P=24, tree=True),  # trees of all sizes
    dict(lead=2, n_max=37, nn=[37, 20], ctx=[64, 200], P=1, tree="odd"),
    dict(lead=0, n_max=3, nn=[3, 2, 0], ctx=[0, 40, 8], P=8, tree="odd"),                  # rows that see nothing
    dict(lead=0, n_max=70, nn=[70, 33, 0], ctx=[0, 100, 5], P=32),                         # causal chunks
]


@pytest.mark.gpu
@pytest.mark.parametrize("size", [dict(dtype=BF16, Dc=512, Dr=64), dict(dtype=F16, Dc=512, Dr=32),
                                  dict(dtype=BF16, Dc=256, Dr=32), dict(dtype=F16, Dc=256, Dr=64)], ids=str)
@pytest.mark.parametrize("Hq", [1, 7, 16, 40, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention(device, size, Hq, shape):
    case = dict(size, Hq=Hq, **SHAPES[shape])
    if Hq * (case["lead"] + case["n_max"]) > 1000:
        case["every"] = 9
    say(case)
    _, c, table, q, w, seen, scale = problem(case)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [dict(dtype=BF16, Dc=512, Dr=64, Dn=128), dict(dtype=F16, Dc=512, Dr=32, Dn=64),
                                  dict(dtype=BF16, Dc=256, Dr=32, Dn=128), dict(dtype=F16, Dc=256, Dr=64, Dn=64)], ids=str)
@pytest.mark.parametrize("Hq", [1, 3, 9])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_prefill(device, size, Hq, shape):
    case = dict(size, Hq=Hq, every=5, **SHAPES[shape])
    say(case)
    _, c, table, q, w, seen, scale = problem(case)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)


@pytest.mark.gpu
def test_prefill_of_a_long_chunk_and_of_fewer_keys_than_there_are(device):
    case = dict(dtype=BF16, Dc=512, Dr=64, Dn=128, Hq=2, lead=0, n_max=515, nn=[515, 300], ctx=[700, 0], P=16, every=101)
    _, c, table, q, w, seen, scale = problem(case)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)
    for keys in (1, 129, 1000):
        out, lse = run_attention(device, case, c, table, q, w, seen, scale, max_keys=keys)
        check_attention(case, c, table, q, w, seen, scale, out, lse, max_keys=keys)


@pytest.mark.gpu
@pytest.mark.parametrize("Dn", [None, 128])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_missing_pages_layers_and_lengths_beyond_the_table(device, dtype, Dn):
    case = dict(dtype=dtype, Dc=512, Dr=64, Hq=5, lead=1, n_max=6, nn=[6, 5, 6], ctx=[150, 90, 40], P=16, tree=True,
                layers=3)
    if Dn:
        case["Dn"] = Dn
    rs, c, table, q, w, seen, scale = problem(case)
    table[0, 2], table[0, 5], table[1, 0], table[1, 1] = -1, c.shape[1], 1 << 30, -(1 << 31)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)
    table[2] = -7                                                 # nothing of this request can be seen
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    case = dict(case, ctx=[150, 2 ** 31 - 1, 1 << 20])            # slots behind the table are not there
    out, lse = run_attention(device, case, c, table, q, w, seen, scale, max_keys=table.shape[1] * 16)
    short = dict(case, ctx=[150, table.shape[1] * 16, table.shape[1] * 16])
    check_attention(short, c, table, q, w, seen, scale, out, lse, max_keys=table.shape[1] * 16)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [2, 16, 128])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("Dn", [None, 64])
def test_unseen_values_stay_out(device, dtype, Hq, Dn):
    """NaN and infinities in nodes off a row's path, and behind its last key."""
    if Dn and Hq == 128:
        Hq = 12
    case = dict(dtype=dtype, Dc=512, Dr=64, Hq=Hq, lead=1, n_max=6, nn=[6], ctx=[70], P=16, tree=True, Dn=Dn)
    if Dn is None:
        del case["Dn"]
    rs, c, table, q, w, seen, scale = problem(case)
    seen[:] = False
    seen[0, np.arange(6), np.arange(6)] = True                    # six children of the root
    for i, value in ((1, math.nan), (3, math.inf), (5, -math.inf)):
        p, o = ref.slot_at(table, c.shape[1], 16, 0, 71 + i)
        c[0, p, o, i::7] = value
        c[0, p, o, 512:] = value
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    clean = c.nan_to_num(0, 0, 0)
    good = [0, 1, 3, 5]                                           # the root and the children that see finite values
    sub = dict(case)
    full = torch.where(torch.isfinite(out), out, torch.zeros_like(out))
    for r in (2, 4, 6):
        full[0, r] = out[0, 1]                                    # not looked at below
        assert torch.isnan(out[0, r].float()).any() or torch.isinf(out[0, r].float()).any()
    for r in good:
        row = seen[0, r - 1] if r else None
        slots = lat.seen_slots(table, c.shape[1], 16, 0, 70, 1, r, 6, row, 1 << 30)
        assert all(torch.isfinite(c[0][ref.slot_at(table, c.shape[1], 16, 0, s)]).all() for s in slots)
        assert torch.isfinite(out[0, r].float()).all()
    twin = run_attention(device, sub, clean, table, q, w, seen, scale)
    for r in good:
        assert torch.equal(out[0, r], twin[0][0, r]) and torch.equal(lse[0, r], twin[1][0, r])


@pytest.mark.gpu
@pytest.mark.parametrize("size", [30.0, 300.0])
def test_large_scores(device, size):
    for dtype in (BF16, F16):
        case = dict(dtype=dtype, Dc=256, Dr=64, Hq=9, lead=1, n_max=2, nn=[2], ctx=[400], P=16, scale=size / 320)
        _, c, table, q, w, seen, scale = problem(case)
        out, lse = run_attention(device, case, c, table, q, w, seen, scale)
        check_attention(case, c, table, q, w, seen, scale, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [16, 12])
@pytest.mark.parametrize("size", [dict(dtype=BF16, Dc=512, Dr=64), dict(dtype=F16, Dc=256, Dr=32)], ids=str)
def test_workgroups_with_thousands_of_keys(device, size, P):
    """So many rows that a workgroup takes all keys of its own, in pages some of
    which are missing (a call of few rows is cut into chunks of 256 keys)."""
    case = dict(size, Hq=128, lead=0, n_max=160, nn=[160, 151], ctx=[3000, 2411], P=P, every=40)
    _, c, table, q, w, seen, scale = problem(case)
    table[0, 5] = table[1, 2100 // P] = table[0, 2900 // P] = -1
    table[1, 1030 // P] = 1 << 30
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)


WIDE = [
    dict(lead=1, n_max=64, nn=[64, 33, 0], ctx=[1500, 31, 2], P=16, tree=True, every=5),   # the benchmark's budget
    dict(lead=1, n_max=64, nn=[63, 64, 32], ctx=[700, 15, 96], P=32, tree="odd", every=5),
    dict(lead=3, n_max=100, nn=[100, 65], ctx=[29, 2111], P=24, tree="odd", every=9),      # four words
    dict(lead=0, n_max=129, nn=[129, 96], ctx=[1, 333], P=12, tree="odd", every=11),       # five, of rows that see nothing, too
    dict(lead=1, n_max=300, nn=[300, 257], ctx=[900, 0], P=16, tree=True, every=41),
    dict(lead=2, n_max=1024, nn=[1024, 800], ctx=[61, 130], P=64, tree="odd", every=151),
]


@pytest.mark.gpu
@pytest.mark.parametrize("size", [dict(dtype=BF16, Dc=512, Dr=64, Hq=128), dict(dtype=F16, Dc=256, Dr=32, Hq=7),
                                  dict(dtype=BF16, Dc=512, Dr=64, Hq=6, Dn=128), dict(dtype=F16, Dc=256, Dr=32, Hq=3, Dn=64)],
                         ids=str)
@pytest.mark.parametrize("shape", range(len(WIDE)))
def test_trees_whose_masks_have_many_words(device, size, shape):
    """Tiles of keys that begin and end inside mask words, in the workgroups'
    own tiles and in split ones."""
    case = dict(size, **WIDE[shape])
    if size["Hq"] == 128:
        case["every"] *= 4
    say(case)
    _, c, table, q, w, seen, scale = problem(case)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("Dn", [None, 64])
def test_strides(device, Dn):
    """Queries, results and slots inside wider buffers give the packed ones'
    results, bit by bit, and nothing beside the results is written."""
    case = dict(dtype=F16, Dc=256, Dr=64, Hq=5, lead=1, n_max=20, nn=[20, 11], ctx=[700, 45], P=8, tree=True, Dn=Dn)
    _, c, table, q, w, seen, scale = problem(case)
    out, _ = run_attention(device, case, c, table, q, w, seen, scale)
    pool = torch.full(c.shape[1:3] + (400,), math.nan, dtype=F16, device=device)
    pool[..., 16:336] = c[0].to(device)
    cache, chunk = bd.LatentCache(pool[..., 16:336], upload(table, device), 64), chunk_on(device, [700, 45], 1, 20, [20, 11], seen)
    dq = torch.full((2, 21, 7, q.shape[-1]), math.nan, dtype=F16, device=device)
    dq[:, :, 1:6] = q.to(device)
    wide = torch.full((2, 21, 8, Dn or 256), SENTINEL, dtype=F16, device=device)
    if Dn is None:
        ws = torch.empty(bd.dt_latent_workspace(cache, chunk, 5), dtype=torch.uint8, device=device)
        bd.dt_latent_attention(cache, chunk, dq[:, :, 1:6], wide[:, :, 2:7], scale, workspace=ws)
    else:
        ws = torch.empty(bd.dt_latent_prefill_workspace(cache, chunk, 5, Dn, 721), dtype=torch.uint8, device=device)
        bd.dt_latent_prefill(cache, chunk, dq[:, :, 1:6], w.to(device), wide[:, :, 2:7], scale, 721, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, :, 2:7].cpu(), out)
    assert (wide[:, :, :2] == SENTINEL).all() and (wide[:, :, 7:] == SENTINEL).all()


@pytest.mark.gpu
def test_many_requests_of_all_lengths(device):
    rs = np.random.RandomState(5)
    ctx = [int(x) for x in 900 * rs.rand(150) ** 3]
    case = dict(dtype=BF16, Dc=256, Dr=32, Hq=16, lead=1, n_max=0, ctx=ctx, P=16)
    _, c, table, q, w, seen, scale = problem(case)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    check_attention(case, c, table, q, w, seen, scale, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("Dn", [None, 64])
def test_cache_beyond_32_bit_offsets(device, Dn):
    """A pool of 2^32 elements: its last pages, which lie behind 2^31 elements."""
    case = dict(dtype=BF16, Dc=256, Dr=64, Hq=6, lead=1, n_max=3, nn=[3, 3], ctx=[45, 20], P=16, tree=True)
    if Dn:
        case["Dn"] = Dn
    rs, c, table, q, w, seen, scale = problem(case)
    pages = 2 ** 32 // (16 * 320)
    free = torch.cuda.mem_get_info()[0]
    if free < 12 << 30:
        pytest.skip("no room for the pool")
    big = torch.zeros(pages, 16, 320, dtype=BF16, device=device)
    shift = pages - c.shape[1]
    big[shift:] = c[0].to(device)
    moved = np.where(table >= 0, table + shift, table).astype(np.int32)
    out, lse = run_attention(device, case, c, table, q, w, seen, scale)
    cache, chunk = bd.LatentCache(big, upload(moved, device), 64), chunk_on(device, [45, 20], 1, 3, [3, 3], seen)
    dq, got = q.to(device), torch.empty(2, 4, 6, Dn or 256, dtype=BF16, device=device)
    if Dn is None:
        ws = torch.empty(bd.dt_latent_workspace(cache, chunk, 6), dtype=torch.uint8, device=device)
        bd.dt_latent_attention(cache, chunk, dq, got, scale, workspace=ws)
    else:
        ws = torch.empty(bd.dt_latent_prefill_workspace(cache, chunk, 6, Dn, 49), dtype=torch.uint8, device=device)
        bd.dt_latent_prefill(cache, chunk, dq, w.to(device), got, scale, 49, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), out)
    x = torch.randn(2, 4, 320, device=device).to(BF16)
    bd.dt_latent_append(cache, chunk, x[..., :256], x[..., 256:])
    torch.cuda.synchronize()
    for b, n in enumerate((45, 20)):
        for r in range(4):
            assert torch.equal(big[int(moved[b, (n + r) // 16]), (n + r) % 16], x[b, r])


@pytest.mark.gpu
def test_calls_in_flight_on_two_streams(device):
    """Both forms on two streams at once, a workspace each, the second in a graph
    that is replayed: every call's results are its own."""
    jobs = []
    for Dn in (None, 128):
        case = dict(dtype=BF16, Dc=512, Dr=64, Hq=16, lead=1, n_max=20, nn=[20, 7, 15], ctx=[4000, 35, 812], P=16, tree=True,
                    Dn=Dn)
        _, c, table, q, w, seen, scale = problem(case)
        cache = bd.LatentCache(c.to(device), upload(table, device), 64)
        chunk = chunk_on(device, case["ctx"], 1, 20, case["nn"], seen)
        dq, dw = q.to(device), None if w is None else w.to(device)
        size = bd.dt_latent_workspace(cache, chunk, 16) if Dn is None else \
            bd.dt_latent_prefill_workspace(cache, chunk, 16, Dn, 4021)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        out = torch.zeros(3, 21, 16, Dn or 512, dtype=BF16, device=device)

        def call(Dn=Dn, cache=cache, chunk=chunk, dq=dq, dw=dw, out=out, ws=ws, scale=scale):
            if Dn is None:
                bd.dt_latent_attention(cache, chunk, dq, out, scale, workspace=ws)
            else:
                bd.dt_latent_prefill(cache, chunk, dq, dw, out, scale, 4021, workspace=ws)
        call()
        torch.cuda.synchronize()
        jobs.append((call, out, out.clone(), torch.cuda.Stream()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jobs[1][0]()
    for _ in range(3):
        for _, out, _, _ in jobs:
            out.zero_()
        torch.cuda.synchronize()
        for call, _, _, stream in jobs:
            with torch.cuda.stream(stream):
                call() if call is jobs[0][0] else graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in jobs:
            assert torch.equal(out, want)


# ---------------------------------------------------------------------------
# commit, and everything together
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    dict(dtype=BF16, D=576, lead=1, n_max=20, nn=[20, 0, 13, 20, 20], ctx=[40, 3, 0, -1, 77], P=16, layers=3),
    dict(dtype=F16, D=288, lead=3, n_max=64, nn=[64, 64], ctx=[11, 300], P=1, layers=1),
], ids=str)
def test_commit(device, case):
    rs = np.random.RandomState(11)
    lead, n_max, nn, ctx, P, D = (case[k] for k in ("lead", "n_max", "nn", "ctx", "P", "D"))
    B, rows, L = len(ctx), lead + n_max, 8
    c, table = lat.make_latents(rs, ctx, rows, P, D, case["dtype"], layers=case["layers"])
    lat.fill_chunk(rs, c, table, ctx, rows)
    parents, _, _ = ref.random_tree(rs, B, n_max, nn)
    tokens = rs.randint(0, 50, (B, n_max)).astype(np.int32)
    target = rs.randint(0, 50, (B, rows)).astype(np.int32)
    for b in range(B):                                            # follow the last child of the last child ...
        cur = -1
        for i in range(max(nn[b], 0)):
            if parents[b, i] == cur and (i + 1 == nn[b] or parents[b, i + 1] != cur):
                target[b, lead + cur] = tokens[b, i]
                cur = i
    dc, dt = c.clone().to(device), 32 if D == 288 else 64
    acc, nodes = (torch.full((B, L), -9, dtype=I32, device=device) for _ in range(2))
    lengths = torch.full((B,), -9, dtype=I32, device=device)
    bd.dt_latent_commit(bd.LatentCache(dc, upload(table, device), dt), chunk_on(device, ctx, lead, n_max, nn),
                        upload(tokens, device), upload(parents, device), upload(target, device), acc, lengths, nodes=nodes)
    torch.cuda.synchronize()
    want = c.clone()
    for b in range(B):
        if ctx[b] < 0:
            assert int(lengths[b]) == 0 and (acc[b] == -1).all()
            continue
        said, path = ref.walk(tokens[b], parents[b], target[b], lead, nn[b], L)
        assert acc[b].tolist() == said + [-1] * (L - len(said)) and int(lengths[b]) == len(said)
        assert nodes[b].tolist() == path + [-1] * (L - len(path))
        for i, n in enumerate(path):
            p, o = ref.slot_at(table, c.shape[1], P, b, ctx[b] + lead + n)
            p1, o1 = ref.slot_at(table, c.shape[1], P, b, ctx[b] + lead + i)
            want[:, p1, o1] = c[:, p, o]
    assert torch.equal(dc.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.gpu
def test_both_forms_agree(device):
    """The absorbed form with the products of the head's weights around it is
    the expanded one."""
    rs = np.random.RandomState(2)
    Hq, Dn, Dc, Dr = 4, 64, 256, 32
    case = dict(dtype=F16, Dc=Dc, Dr=Dr, Dn=Dn, Hq=Hq, lead=0, n_max=90, nn=[90, 41], ctx=[33, 200], P=16)
    _, c, table, q, w, seen, scale = problem(case)
    made, ml = run_attention(device, case, c, table, q, w, seen, scale)
    ww = w.double()
    absorbed = torch.cat((torch.einsum("brhn,hnc->brhc", q[..., :Dn].double(), ww[:, :Dn]), q[..., Dn:].double()), -1).half()
    one = {k: v for k, v in case.items() if k != "Dn"}
    out, ol = run_attention(device, one, c, table, absorbed, None, seen, scale)
    back = torch.einsum("brhc,hnc->brhn", out.double(), ww[:, Dn:])
    for b, n in enumerate((90, 41)):
        # a few roundings of 2^-11 on each side, of scores up to a few units and results of about one
        assert (ml[b, :n] - ol[b, :n]).abs().max() < 64 * 2.0 ** -11
        assert (made[b, :n].double() - back[b, :n]).abs().max() < 64 * 2.0 ** -11


@pytest.mark.gpu
def test_round_as_it_is_used_and_captured(device):
    """Verification rounds of a tree over latents: append, attention, drawn
    tokens, commit; eager, and captured and replayed with other lengths, on a
    stream of its own."""
    rs = np.random.RandomState(8)
    B, Hq, Dc, Dr, P, n_max, V = 3, 8, 256, 64, 16, 12, 500
    ctx0 = [37, 0, 64]
    parents, depths, seen = ref.random_tree(rs, B, n_max, [12, 12, 12])
    c, table = lat.make_latents(rs, ctx0, 1 + n_max + 60, P, Dc + Dr, BF16)
    tokens = rs.randint(0, V, (B, n_max)).astype(np.int32)
    g = torch.Generator().manual_seed(1)
    steps = [dict(x=torch.randn(B, 1 + n_max, Dc + Dr, generator=g).to(BF16),
                  q=torch.randn(B, 1 + n_max, Hq, Dc + Dr, generator=g).to(BF16),
                  logits=torch.randn(B, 1 + n_max, V, generator=g) * 3, u=torch.rand(B, 1 + n_max, generator=g),
                  nn=torch.from_numpy(rs.randint(0, n_max + 1, B).astype(np.int32))) for _ in range(4)]
    for s in steps:                                               # tokens of the tree are likely
        s["logits"].scatter_add_(2, torch.from_numpy(tokens).long()[:, None].expand(B, 1 + n_max, n_max),
                                 torch.full((B, 1 + n_max, n_max), 6.0))
    freqs = torch.from_numpy(10000.0 ** (-np.arange(0, Dr, 2) / Dr)).to(device)

    class Side:
        def __init__(self):
            self.c = c.clone().to(device)
            self.cache = bd.LatentCache(self.c, upload(table, device), Dr)
            self.ctx = torch.tensor(ctx0, dtype=I32, device=device)
            self.nn = torch.zeros(B, dtype=I32, device=device)
            self.chunk = bd.Chunk(self.ctx, 1, n_max, self.nn, upload(ref.pack_bits(seen), device), upload(depths, device))
            self.x, self.q = (torch.zeros_like(steps[0][k], device=device) for k in ("x", "q"))
            self.logits, self.u = (torch.zeros_like(steps[0][k], device=device) for k in ("logits", "u"))
            self.tokens, self.parents = upload(tokens, device), upload(parents, device)
            self.out = torch.zeros(B, 1 + n_max, Hq, Dc, dtype=BF16, device=device)
            self.target = torch.zeros(B, 1 + n_max, dtype=I32, device=device)
            self.logp = torch.zeros(B, 1 + n_max, device=device)
            self.acc, self.len = torch.zeros(B, 6, dtype=I32, device=device), torch.zeros(B, dtype=I32, device=device)
            self.ws = torch.empty(bd.dt_latent_workspace(self.cache, self.chunk, Hq), dtype=torch.uint8, device=device)
            self.ws2 = torch.empty(max(bd.dt_sample_workspace(self.logits), 16), dtype=torch.uint8, device=device)
            self.heat = torch.tensor([0.7, 1.0, 0.0], device=device)
            self.k = torch.tensor([20, 0, 0], dtype=I32, device=device)
            self.p = torch.tensor([0.9, 0.95, 1.0], device=device)

        def load(self, s):
            for name in ("x", "q", "logits", "u", "nn"):
                getattr(self, name).copy_(s[name])

        def step(self):
            bd.dt_latent_append(self.cache, self.chunk, self.x[..., :Dc], self.x[..., Dc:], q_rot=self.q[..., Dc:],
                                q_out=self.q[..., Dc:], freqs=freqs)
            bd.dt_latent_attention(self.cache, self.chunk, self.q, self.out, 0.07, workspace=self.ws)
            bd.dt_sample_rows(self.logits, self.u, self.target, temperature=self.heat, top_k=self.k, top_p=self.p,
                              logp=self.logp, lead=1, n_nodes=self.nn, workspace=self.ws2)
            bd.dt_latent_commit(self.cache, self.chunk, self.tokens, self.parents, self.target, self.acc, self.len)
            self.ctx += self.len

        def state(self):
            return [t.cpu().clone() for t in (self.c.view(torch.int16), self.ctx, self.out, self.target, self.logp, self.acc)]

    eager, graphed = Side(), Side()
    want = []
    for s in steps:
        eager.load(s)
        eager.step()
        torch.cuda.synchronize()
        want.append(eager.state())
        for b in range(B):                                        # the drawn tokens are the definition's
            for r in range(1 + int(s["nn"][b])):
                t, lp, near = lat.draw_row(s["logits"][b, r].numpy(), float(s["u"][b, r]), float(eager.heat[b]),
                                           int(eager.k[b]), float(eager.p[b]))
                assert near > 1e-11 and int(want[-1][3][b, r]) == t
    assert int(want[-1][1].sum()) > sum(ctx0) + 4 * B             # trees were accepted
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    graphed.load(steps[0])
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graphed.step()                                            # (undone below)
    torch.cuda.synchronize()
    graphed.c.copy_(c)
    graphed.ctx.copy_(torch.tensor(ctx0, dtype=I32))
    for t in (graphed.out, graphed.target, graphed.logp, graphed.acc):
        t.zero_()
    with torch.cuda.graph(graph):
        graphed.step()
    for s, w in zip(steps, want):
        graphed.load(s)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(graphed.state(), w):
            assert torch.equal(x, y)
