"""The verification pass (dt_kv_append, dt_tree_attention, dt_process_logits,
dt_commit_path) against its definitions in 64 bits (pass_ref.py)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import pass_ref as ref
from draft_tree_construction_dt_amd import synth

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SENTINEL = 7.0


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# host side: frequencies and refusals (no GPU)
# ---------------------------------------------------------------------------

def test_rope_frequencies_plain_and_linear():
    f, s = bd.dt_rope_frequencies(128, 10000.0)
    want = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    assert s == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14, atol=0)
    f, s = bd.dt_rope_frequencies(64, 500000.0, bd.DT_ROPE_LINEAR, factor=4.0)
    assert s == 1.0 and np.allclose(f.numpy(), 500000.0 ** (-np.arange(0, 64, 2) / 64) / 4, rtol=1e-14, atol=0)


def test_rope_frequencies_by_wavelength():
    f, s = bd.dt_rope_frequencies(128, 500000.0, bd.DT_ROPE_WAVELENGTH, factor=8.0, low=1.0, high=4.0, original=8192)
    assert s == 1.0
    for i, got in enumerate(f.tolist()):
        plain = 500000.0 ** (-2 * i / 128)
        lam = 2 * math.pi / plain
        if lam > 8192:
            want = plain / 8
        elif lam < 2048:
            want = plain
        else:
            k = (8192 / lam - 1) / 3
            want = (1 - k) * plain / 8 + k * plain
        assert got == pytest.approx(want, rel=1e-12)


def test_rope_frequencies_yarn():
    f, s = bd.dt_rope_frequencies(128, 1e6, bd.DT_ROPE_YARN, factor=4.0, low=1.0, high=32.0, original=32768)
    assert s == pytest.approx(0.1 * math.log(4.0) + 1, rel=1e-7)
    lo = math.floor(128 * math.log(32768 / (32 * 2 * math.pi)) / (2 * math.log(1e6)))
    hi = math.ceil(128 * math.log(32768 / (2 * math.pi)) / (2 * math.log(1e6)))
    for i, got in enumerate(f.tolist()):
        plain = 1e6 ** (-2 * i / 128)
        k = min(max((i - lo) / (hi - lo), 0), 1)
        assert got == pytest.approx(plain / 4 * k + plain * (1 - k), rel=1e-12)
    assert bd.dt_rope_frequencies(128, 1e6, bd.DT_ROPE_YARN, factor=0.5, original=32768)[1] == 1.0


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=15), dict(rot_dim=-2), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
    dict(factor=0.0), dict(factor=math.nan), dict(kind=4), dict(kind=-1),
    dict(kind=2, low=0.0), dict(kind=2, low=4.0, high=4.0), dict(kind=3, original=0.0), dict(kind=3, high=math.inf),
])
def test_rope_frequencies_refusals(kw):
    args = dict(rot_dim=64, base=10000.0)
    args.update(kw)
    with pytest.raises(bd.DtError) as e:
        bd.dt_rope_frequencies(**args)
    assert e.value.status == bd.DT_ERR_INVALID_ARG


FAKE = 0x100000
BAD, LIMIT, WORK = bd.DT_ERR_INVALID_ARG, bd.DT_ERR_UNSUPPORTED, bd.DT_ERR_WORKSPACE


def _struct(cls, base, kw):
    base = dict(base)
    base.update(kw)
    s = cls()
    for k, v in base.items():
        setattr(s, k, v)
    return s


def _kv(**kw):
    return _struct(bd._KVCache, dict(k=FAKE, v=FAKE, page_table=FAKE, layer_stride=1 << 20, page_stride=16384,
                                     slot_stride=1024, head_stride=128, layers=2, num_pages=9, page_size=16,
                                     max_pages=8, Hkv=8, D=128, dtype=bd.DT_DTYPE_BF16), kw)


def _chunk(**kw):
    return _struct(bd._Chunk, dict(B=2, lead=1, n_max=8, ctx_len=FAKE), kw)


def _append(**kw):
    return _struct(bd._AppendParams, dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, q_stride=6144, k_stride=6144,
                                          v_stride=6144, q_out_stride=6144, Hq=32, eps=1e-6, freqs=FAKE, rot_dim=64,
                                          rot_scale=1.0), kw)


def _attention(**kw):
    return _struct(bd._AttentionParams, dict(q=FAKE, out=2 * FAKE, q_stride=4096, out_stride=4096, Hq=32, scale=0.1,
                                             workspace=FAKE, workspace_bytes=1 << 40), kw)


def _logits(**kw):
    return _struct(bd._LogitsParams, dict(logits=FAKE, out=FAKE, B=2, lead=4, n_max=3, V=1000, dtype=1), kw)


def _commit(**kw):
    return _struct(bd._CommitParams, dict(tokens=FAKE, parents=FAKE, target=FAKE, L=9, accepted=FAKE, lengths=FAKE),
                   kw)


BAD_CACHES = [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(page_table=None), BAD), (dict(k=FAKE + 8), BAD),
    (dict(v=FAKE + 2), BAD), (dict(page_table=FAKE + 2), BAD), (dict(layers=0), BAD), (dict(num_pages=0), BAD),
    (dict(page_size=0), BAD), (dict(max_pages=0), BAD), (dict(Hkv=0), BAD), (dict(D=0), BAD), (dict(dtype=0), BAD),
    (dict(dtype=3), BAD), (dict(layer_stride=4), BAD), (dict(page_stride=-8), BAD), (dict(slot_stride=12), BAD),
    (dict(head_stride=1), BAD), (dict(D=96), LIMIT), (dict(D=32), LIMIT), (dict(Hkv=8192), LIMIT),
    (dict(page_size=1 << 16, max_pages=1 << 15), LIMIT),
]
BAD_CHUNKS = [
    (dict(B=-1), BAD), (dict(lead=-1), BAD), (dict(n_max=-1), BAD), (dict(lead=0, n_max=0), BAD),
    (dict(ctx_len=None), BAD), (dict(ctx_len=FAKE + 1), BAD), (dict(n_nodes=FAKE + 2), BAD),
    (dict(B=65536), LIMIT), (dict(lead=65530), LIMIT), (dict(B=4096, n_max=4096), LIMIT),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(kw, status):
    lib, c = bd._load(), _chunk()
    if "Hkv" in kw and kw["Hkv"] > 4096:
        p, a = _append(Hq=1), _attention(Hq=8192)
    else:
        p, a = _append(), _attention()
    kv = _kv(**kw)
    assert lib.dt_kv_append(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == status
    assert lib.dt_tree_attention(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(a)) == status
    m = _commit()
    assert lib.dt_commit_path(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(m)) == status


@pytest.mark.parametrize("kw,status", BAD_CHUNKS)
def test_bad_chunks_are_refused(kw, status):
    lib, kv, c, p, a, m = bd._load(), _kv(), _chunk(**kw), _append(), _attention(), _commit()
    assert lib.dt_kv_append(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == status
    assert lib.dt_tree_attention(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(a)) == status
    assert lib.dt_commit_path(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(m)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(q=None), BAD), (dict(q_out=None), BAD), (dict(q=FAKE + 8), BAD),
    (dict(k_stride=1020), BAD), (dict(k_stride=512), BAD), (dict(q_stride=2048), BAD), (dict(v_stride=0), BAD),
    (dict(q_out_stride=4096), BAD),                    # q itself, at another stride
    (dict(Hq=0), BAD), (dict(Hq=5000), LIMIT), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
    (dict(rot_dim=-16), BAD), (dict(rot_dim=144), BAD), (dict(rot_dim=24), LIMIT), (dict(freqs=None), BAD),
    (dict(freqs=FAKE + 4), BAD), (dict(rot_scale=math.inf), BAD), (dict(layer=2), BAD), (dict(layer=-1), BAD),
    (dict(q_norm=FAKE + 2), BAD), (dict(k_norm=FAKE + 8), BAD),
])
def test_append_refusals(kw, status):
    kv, c, p = _kv(), _chunk(), _append(**kw)
    assert bd._load().dt_kv_append(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(out=FAKE), BAD), (dict(q=FAKE + 8), BAD),
    (dict(q_stride=2048), BAD), (dict(out_stride=4100), BAD), (dict(Hq=0), BAD), (dict(Hq=12), BAD),
    (dict(Hq=8192), LIMIT), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD),
    (dict(scale=math.inf), BAD), (dict(lse=FAKE + 2), BAD), (dict(layer=2), BAD), (dict(layer=-1), BAD),
    (dict(workspace=None), WORK), (dict(workspace=FAKE + 4), WORK), (dict(workspace_bytes=16), WORK),
])
def test_attention_refusals(kw, status):
    kv, c, p = _kv(), _chunk(), _attention(**kw)
    assert bd._load().dt_tree_attention(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == status


def test_attention_limits_of_a_call():
    kv, c, p = _kv(Hkv=1), _chunk(B=65535, lead=1, n_max=40), _attention(Hq=4096, q_stride=1 << 20,
                                                                         out_stride=1 << 20)
    lib = bd._load()
    assert lib.dt_tree_attention(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == LIMIT
    assert lib.dt_attention_workspace(ctypes.byref(kv), ctypes.byref(c), 4096) == 0
    assert lib.dt_attention_workspace(None, ctypes.byref(c), 8) == 0
    ok = _chunk()
    assert lib.dt_attention_workspace(ctypes.byref(kv), ctypes.byref(ok), 8) > 0
    assert lib.dt_attention_workspace(ctypes.byref(_kv()), ctypes.byref(ok), 12) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), BAD), (dict(out=None), BAD), (dict(out=FAKE + 8), BAD), (dict(B=-1), BAD), (dict(V=0), BAD),
    (dict(lead=-1), BAD), (dict(n_max=-1), BAD), (dict(lead=0, n_max=0), BAD), (dict(dtype=2), BAD),
    (dict(history=FAKE, history_max=8), BAD), (dict(history_max=-1), BAD), (dict(n_bias=-1), BAD),
    (dict(node_tokens=FAKE), BAD), (dict(bias_ids=FAKE, n_bias=2), BAD), (dict(allow=FAKE), BAD),
    (dict(allow=FAKE, allow_rows=13), BAD), (dict(n_nodes=FAKE + 2), BAD), (dict(presence=FAKE + 1), BAD),
    (dict(B=65536), LIMIT), (dict(V=1 << 26), LIMIT), (dict(n_bias=65535), LIMIT),
    (dict(node_tokens=FAKE, node_mask=FAKE, n_max=1025), LIMIT), (dict(lead=65536), LIMIT),
])
def test_logits_refusals(kw, status):
    p = _logits(**kw)
    assert bd._load().dt_process_logits(ctypes.byref(p)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=None), BAD), (dict(parents=None), BAD), (dict(target=None), BAD), (dict(accepted=None), BAD),
    (dict(lengths=None), BAD), (dict(L=0), BAD), (dict(nodes=FAKE + 2), BAD),
])
def test_commit_refusals(kw, status):
    kv, c, p = _kv(), _chunk(), _commit(**kw)
    assert bd._load().dt_commit_path(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == status


def test_commit_refuses_chunks_without_a_root_and_huge_trees():
    lib, kv, p = bd._load(), _kv(), _commit()
    for c, status in ((_chunk(lead=0), BAD), (_chunk(n_max=1025), LIMIT)):
        assert lib.dt_commit_path(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(p)) == status


def test_empty_batches_and_null_structs():
    lib, kv, c = bd._load(), _kv(), _chunk(B=0, ctx_len=None)
    assert lib.dt_kv_append(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(_append(k=None, v=None))) == bd.DT_OK
    assert lib.dt_tree_attention(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(_attention(q=None))) == bd.DT_OK
    assert lib.dt_process_logits(ctypes.byref(_logits(B=0, logits=None))) == bd.DT_OK
    assert lib.dt_commit_path(ctypes.byref(kv), ctypes.byref(c), ctypes.byref(_commit(target=None))) == bd.DT_OK
    full = _chunk()
    assert lib.dt_kv_append(None, ctypes.byref(full), ctypes.byref(_append())) == BAD
    assert lib.dt_kv_append(ctypes.byref(kv), None, ctypes.byref(_append())) == BAD
    assert lib.dt_kv_append(ctypes.byref(kv), ctypes.byref(full), None) == BAD
    assert lib.dt_tree_attention(None, ctypes.byref(full), ctypes.byref(_attention())) == BAD
    assert lib.dt_tree_attention(ctypes.byref(kv), ctypes.byref(full), None) == BAD
    assert lib.dt_process_logits(None) == BAD
    assert lib.dt_commit_path(ctypes.byref(kv), None, ctypes.byref(_commit())) == BAD


def test_binding_checks_tensors():
    k = torch.zeros(4, 16, 2, 64, dtype=BF16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    kv = bd.KVCache(k, k.clone(), table)
    assert (kv.layers, kv.Hkv, kv.D) == (1, 2, 64)
    for bad in (dict(v=k.float()), dict(v=torch.zeros(4, 16, 2, 128, dtype=BF16)), dict(page_table=table.long()),
                dict(k=k[..., ::2], v=k[..., ::2]), dict(k=k.float(), v=k.float()),
                dict(v=torch.zeros(4, 2, 16, 64, dtype=BF16).transpose(1, 2))):
        with pytest.raises(bd.DtError):
            bd.KVCache(**dict(dict(k=k, v=k.clone(), page_table=table), **bad))
    ctx = torch.zeros(2, dtype=torch.int32)
    for bad in (dict(ctx_len=ctx.long()), dict(n_nodes=torch.zeros(3, dtype=torch.int32)),
                dict(n_max=40, mask=torch.zeros(2, 40, 1, dtype=torch.int32)),
                dict(n_max=4, depths=torch.zeros(2, 3, dtype=torch.int32))):
        with pytest.raises(bd.DtError):
            bd.Chunk(**dict(dict(ctx_len=ctx), **bad))
    chunk = bd.Chunk(ctx, lead=3)
    q = torch.zeros(2, 3, 4, 64, dtype=BF16)
    out = torch.zeros_like(q)
    for bad in (dict(q=q.half()), dict(q=q[:, :2]), dict(q=q[:1]), dict(out=out[:, :, :2]), dict(q=q.transpose(0, 1)),
                dict(q=torch.zeros(2, 4, 4, 64, dtype=BF16)[:, :3]), dict(lse=torch.zeros(2, 3, 3)),
                dict(q=torch.zeros(2, 3, 64, 4, dtype=BF16).transpose(2, 3))):
        with pytest.raises(bd.DtError):
            bd.dt_tree_attention(kv, chunk, **dict(dict(q=q, out=out), **bad))
    with pytest.raises(bd.DtError):
        bd.dt_kv_append(kv, chunk, q[:, :, :3], q[:, :, :2])
    with pytest.raises(bd.DtError):
        bd.dt_kv_append(bd.KVCache(k, k.clone(), table[:1]), chunk, q[:, :, :2], q[:, :, :2])
    none = bd.KVCache(k, k.clone(), table[:0]), bd.Chunk(ctx[:0], lead=3)       # an empty batch: nothing is launched
    bd.dt_tree_attention(*none, q[:0], out[:0], workspace=None if bd.dt_attention_workspace(*none, 4) == 0 else
                         torch.empty(bd.dt_attention_workspace(*none, 4), dtype=torch.uint8))
    bd.dt_kv_append(*none, q[:0, :, :2], q[:0, :, :2], q=q[:0], q_out=out[:0])
    bd.dt_process_logits(torch.zeros(0, 3, 50), torch.zeros(0, 3, 50))
    bd.dt_commit_path(*none, None, None, torch.zeros(0, 3, dtype=torch.int32), torch.zeros(0, 4, dtype=torch.int32),
                      torch.zeros(0, dtype=torch.int32))
    x = torch.zeros(2, 3, 50)
    for bad in (dict(out=x.bfloat16()), dict(history=torch.zeros(2, 5)), dict(frequency=torch.zeros(3)),
                dict(lead=4), dict(allow=torch.zeros(6, 1, dtype=torch.int32)),
                dict(out=torch.zeros(2, 3, 100)[..., ::2]), dict(logits=x.half(), out=x.half())):
        with pytest.raises(bd.DtError):
            bd.dt_process_logits(**dict(dict(logits=x, out=x.clone()), **bad))
    with pytest.raises(bd.DtError):
        bd.dt_commit_path(None, chunk, None, None, torch.zeros(2, 2, dtype=torch.int32),
                          torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


# ---------------------------------------------------------------------------
# problems
# ---------------------------------------------------------------------------

def make_cache(rs, ctx, rows, P, Hkv, D, dtype, layers=1, layout="slots", spare=3, width=0):
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
    gen = torch.Generator().manual_seed(int(rs.randint(1 << 30)))
    if layout == "slots":
        k, v = (torch.randn(layers, pages, P, Hkv, D, generator=gen).to(dtype) for _ in range(2))
    elif layout == "heads":
        k, v = (torch.randn(layers, pages, Hkv, P, D, generator=gen).to(dtype).transpose(2, 3) for _ in range(2))
    else:                                        # keys and values of a page side by side
        both = torch.randn(layers, pages, 2, P, Hkv, D, generator=gen).to(dtype)
        k, v = both[:, :, 0], both[:, :, 1]
    used = np.zeros((pages, P), bool)
    for b, c in enumerate(ctx):
        for s in range(max(c, 0)):
            used[table[b, s // P], s % P] = True
    free = torch.from_numpy(~used)
    k[:, free] = math.nan
    v[:, free] = math.nan
    return k, v, table


def to_device(t, device):
    """A copy on the device with the same strides."""
    if t is None:
        return None
    t = torch.from_numpy(t) if isinstance(t, np.ndarray) else t
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=device)
    return out.copy_(t)


def pair_on_device(k, v, device):
    if k.untyped_storage().data_ptr() == v.untyped_storage().data_ptr():
        both = torch.stack((k, v), 2).contiguous().to(device)
        return both[:, :, 0], both[:, :, 1]
    return to_device(k, device), to_device(v, device)


# ---------------------------------------------------------------------------
# dt_kv_append
# ---------------------------------------------------------------------------

APPEND = [
    # ctx, lead, n_max, n_nodes, Hq, Hkv, D, P, dtype, rot, interleaved, norm, layout
    ([0], 1, 0, None, 4, 1, 128, 16, BF16, 128, False, True, "slots"),
    ([5, 0, 130, 31], 1, 9, [9, 0, 4, 7], 8, 2, 128, 16, BF16, 128, False, True, "slots"),
    ([3, 17, -1], 2, 33, [33, 1, 5], 7, 1, 64, 1, F16, 32, True, False, "heads"),
    ([100003, 7], 0, 21, [21, 13], 5, 5, 256, 24, BF16, 64, False, True, "both"),
    ([70001], 0, 6, None, 3, 3, 64, 64, F16, 16, True, True, "slots"),
    ([11, 12], 3, 5, [5, 2], 16, 4, 256, 16, F16, 256, True, True, "heads"),
    ([40], 1, 5, [5], 2, 2, 128, 8, BF16, 0, False, False, "slots"),
    ([9, 1], 1, 4, [-3, 90], 40, 8, 64, 16, BF16, 64, False, True, "slots"),
    ([1 << 20], 1, 2, [2], 1, 1, 128, 256, F16, 128, False, False, "slots"),
    ([300, 2, 64, 15, 16], 1, 64, [64, 60, 0, 3, 64], 32, 8, 128, 16, BF16, 128, False, True, "slots"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(device, case):
    ctx, lead, n_max, nn, Hq, Hkv, D, P, dtype, rot, inter, norm, layout = APPEND[case]
    say(f"[case] append {case}: {APPEND[case]}")
    rs = np.random.RandomState(100 + case)
    B, rows = len(ctx), lead + n_max
    far = max(ctx) > 2000                        # only the last pages exist; the rest of the table is empty
    short = [c % 97 for c in ctx] if far else ctx
    k, v, table = make_cache(rs, short, rows, P, Hkv, D, dtype, layers=2, layout=layout)
    if far:
        big = np.full((B, max((c + rows + P - 1) // P for c in ctx)), -1, np.int32)
        order = iter(rs.permutation(k.shape[1]))
        for b, c in enumerate(ctx):
            for i in range(c // P, (c + rows - 1) // P + 1):
                big[b, i] = next(order)
        table = big
    tree = nn is not None and lead > 0
    clamped = [min(max(n, 0), n_max) for n in nn] if nn is not None else None
    depths = ref.random_tree(rs, B, n_max, clamped)[1] if tree else None
    qkv = torch.from_numpy(rs.randn(B, rows, Hq + 2 * Hkv, D).astype(np.float32)).to(dtype)
    wq, wk = (torch.from_numpy(1 + 0.3 * rs.randn(D).astype(np.float32)).to(dtype) if norm else None for _ in "qk")
    freqs, scale = (bd.dt_rope_frequencies(rot, 1e6, bd.DT_ROPE_YARN if inter else bd.DT_ROPE_NONE, factor=4.0,
                                           original=4096) if rot else (None, 1.0))
    dk, dv = pair_on_device(k, v, device)
    i32 = dict(dtype=torch.int32, device=device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    chunk = bd.Chunk(torch.tensor(ctx, **i32), lead, n_max, None if nn is None else torch.tensor(nn, **i32),
                     depths=to_device(depths, device))
    dq = qkv.to(device)
    q_out = torch.full((B, rows, Hq, D), SENTINEL, dtype=dtype, device=device)
    layer = case % 2
    bd.dt_kv_append(kv, chunk, dq[:, :, Hq:Hq + Hkv], dq[:, :, Hq + Hkv:], q=dq[:, :, :Hq], q_out=q_out,
                    q_norm=to_device(wq, device), k_norm=to_device(wk, device), eps=1e-6,
                    freqs=to_device(freqs, device), interleaved=inter, rot_scale=scale, layer=layer)
    torch.cuda.synchronize()
    got_q, got_k, got_v = q_out.cpu().double().numpy(), dk.cpu(), dv.cpu()
    x = qkv.double().numpy()
    f = None if freqs is None else freqs.numpy()
    w64 = [None if w is None else w.double().numpy() for w in (wq, wk)]
    for b in range(B):
        live = ref.rows_of(b, ctx, lead, n_max, nn)
        assert np.all(got_q[b, live:] == SENTINEL)
        for r in range(live):
            pos = ctx[b] + r
            if depths is not None and r >= lead:
                pos = ctx[b] + lead - 1 + int(depths[b, r - lead])
            at = ref.slot_at(table, k.shape[1], P, b, ctx[b] + r)
            for h in range(Hq + Hkv):
                want, size = ref.append_head(x[b, r, h], w64[0 if h < Hq else 1], 1e-6, pos, f, inter, scale)
                have = got_q[b, r, h] if h < Hq else got_k[layer, at[0], at[1], h - Hq].double().numpy()
                tol = ref.append_tolerance(want, size, dtype)
                assert np.all(np.abs(have - want) <= tol), (b, r, h, np.max(np.abs(have - want) - tol))
            assert torch.equal(got_v[layer, at[0], at[1]], qkv[b, r, Hq + Hkv:])
            for cache, was in ((got_k, k), (got_v, v)):
                was[layer, at[0], at[1]] = cache[layer, at[0], at[1]]     # checked above
    bits = torch.int16
    assert torch.equal(got_k.contiguous().view(bits), k.contiguous().view(bits)), "a key outside the chunk changed"
    assert torch.equal(got_v.contiguous().view(bits), v.contiguous().view(bits)), "a value outside the chunk changed"


@pytest.mark.gpu
def test_append_in_place_without_queries_and_bad_pages(device):
    rs = np.random.RandomState(5)
    ctx, lead, Hq, Hkv, D, P = [6, 30], 4, 6, 2, 64, 4
    k, v, table = make_cache(rs, ctx, lead, P, Hkv, D, BF16)
    table[0, 2] = k.shape[1]                     # slots 8..11 of request 0: no such page
    table = table[:, :9].copy()                  # request 1's slots 32, 33: page 8; none behind
    x = torch.from_numpy(rs.randn(2, lead, Hq + 2 * Hkv, D).astype(np.float32)).to(BF16).to(device)
    freqs = bd.dt_rope_frequencies(D, 10000.0)[0].to(device)
    ctx_len = torch.tensor([6, 33], dtype=torch.int32, device=device)
    outs = []
    for way in ("out", "in place", "no queries"):
        dk, dv = pair_on_device(k, v, device)
        kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
        q = x[:, :, :Hq].contiguous()
        q_out = q if way == "in place" else torch.empty_like(q)
        kw = {} if way == "no queries" else dict(q=q, q_out=q_out)
        bd.dt_kv_append(kv, bd.Chunk(ctx_len, lead), x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], freqs=freqs, **kw)
        torch.cuda.synchronize()
        outs.append((q_out.cpu(), dk.cpu().view(torch.int16), dv.cpu().view(torch.int16)))
    assert torch.equal(outs[0][0], outs[1][0])
    for i in (1, 2):
        assert torch.equal(outs[0][i], outs[1][i]) and torch.equal(outs[0][i], outs[2][i])
    changed = (outs[0][2] != v.view(torch.int16)).flatten(3).any(-1)[0].nonzero().tolist()
    want = [[int(table[0, 1]), 2], [int(table[0, 1]), 3]] + [[int(table[1, 8]), o] for o in (1, 2, 3)]
    assert sorted(changed) == sorted(want)


# ---------------------------------------------------------------------------
# dt_tree_attention
# ---------------------------------------------------------------------------

ATTEND = [
    # ctx, lead, n_max, n_nodes, mask kind, Hq, Hkv, D, P, dtype, layout
    ([0], 1, 0, None, None, 1, 1, 64, 16, BF16, "slots"),
    ([0, 1, 63, 64, 65, 200], 1, 0, None, None, 8, 2, 128, 16, BF16, "slots"),
    ([5, -1, 300], 1, 0, None, None, 7, 1, 128, 1, F16, "heads"),
    ([1000, 0, 31], 1, 0, None, None, 16, 2, 256, 24, BF16, "both"),
    ([0], 0, 1, None, None, 2, 2, 128, 16, BF16, "slots"),
    ([0, 7, 130], 0, 37, [37, 0, 20], None, 4, 1, 128, 16, BF16, "slots"),
    ([64, 100], 0, 150, [150, 129], None, 6, 2, 64, 64, F16, "heads"),
    ([33], 0, 70, None, None, 5, 1, 256, 32, F16, "slots"),
    ([100, 0, 259, 63], 1, 64, [64, 60, 0, 33], "tree", 8, 2, 128, 16, BF16, "slots"),
    ([129], 1, 64, [64], "tree", 32, 8, 128, 16, BF16, "both"),
    ([40, 513], 2, 100, [100, 97], "tree", 7, 1, 64, 32, F16, "slots"),
    ([0, 20], 0, 45, [45, 30], "random", 4, 2, 128, 8, BF16, "slots"),     # rows that see nothing
    ([0, 0], 0, 65, [65, 64], "none", 3, 1, 64, 16, F16, "slots"),         # no bit set anywhere
    ([77, 500], 3, 256, [256, 200], "random", 14, 2, 64, 32, BF16, "heads"),
    ([10, 200], 1, 33, [33, 30], "tree", 12, 3, 256, 16, BF16, "slots"),
    ([2500, 1], 1, 16, [16, 16], "tree", 2, 2, 128, 256, BF16, "slots"),
    ([4000], 1, 0, None, None, 4, 4, 128, 16, F16, "slots"),
]


def attention_problem(case, seed=0, spec=None):
    ctx, lead, n_max, nn, kind, Hq, Hkv, D, P, dtype, layout = spec or ATTEND[case]
    rs = np.random.RandomState(900 + case + 1000 * seed)
    B, rows = len(ctx), lead + n_max
    whole = [c + ref.rows_of(b, ctx, lead, n_max, nn) if c >= 0 else -1 for b, c in enumerate(ctx)]
    k, v, table = make_cache(rs, whole, 0, P, Hkv, D, dtype, layers=2, layout=layout, width=1)
    seen = None
    if kind == "tree":
        seen = ref.random_tree(rs, B, n_max, nn, width=8)[2]
    elif kind == "random":
        seen = rs.rand(B, n_max, n_max) < 0.2          # bits behind n_nodes are set too
        seen[:, ::5] = False
    elif kind == "none":
        seen = np.zeros((B, n_max, n_max), bool)
    q = torch.from_numpy(rs.randn(B, rows, Hq, D).astype(np.float32)).to(dtype)
    return k, v, table, seen, q


def run_attention(device, ctx, lead, n_max, nn, seen, q, kv, layer, lse=True, scale=None, mask=None, stream=None):
    i32 = dict(dtype=torch.int32, device=device)
    if seen is not None:
        mask = torch.from_numpy(ref.pack_bits(seen)).to(device)
    chunk = bd.Chunk(torch.tensor(ctx, **i32), lead, n_max, None if nn is None else torch.tensor(nn, **i32), mask=mask)
    dq = to_device(q, device)
    out = torch.full(q.shape, SENTINEL, dtype=q.dtype, device=device)
    L = torch.full(q.shape[:3], SENTINEL, device=device) if lse else None
    ws = torch.empty(max(bd.dt_attention_workspace(kv, chunk, q.shape[2]), 16), dtype=torch.uint8, device=device)
    ws.fill_(255)                                # NaN in whatever the workspace holds before
    bd.dt_tree_attention(kv, chunk, dq, out, lse=L, layer=layer, workspace=ws, scale=scale, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().double().numpy(), None if L is None else L.cpu().double().numpy()


def check_attention(ctx, lead, n_max, nn, seen, q, k, v, table, P, got, lse, scale, dtype, layer, rows=None):
    B, Hq, Hkv = len(ctx), q.shape[2], k.shape[3]
    q64 = q.double().numpy()
    pages = k.shape[1]
    for b in range(B):
        live = ref.rows_of(b, ctx, lead, n_max, nn)
        assert np.all(got[b, live:] == SENTINEL) and np.all(lse[b, live:] == SENTINEL)
        for r in range(live) if rows is None else rows:
            slots = ref.visible(ctx[b], lead, r, live - lead, None if seen is None or r < lead else seen[b, r - lead])
            at = [x for x in (ref.slot_at(table, pages, P, b, s) for s in slots) if x is not None]
            pg, off = (torch.tensor([a[i] for a in at], dtype=torch.long) for i in (0, 1))
            K, V = k[layer, pg, off].double().numpy(), v[layer, pg, off].double().numpy()
            for h in range(Hq):
                g = h // (Hq // Hkv)
                want, wl, spread, slack, vmax = ref.attend_row(q64[b, r, h], K[:, g], V[:, g], scale)
                tol = ref.attend_tolerance(want, spread, slack, vmax, len(at), dtype)
                err = np.abs(got[b, r, h] - want)
                assert np.all(err <= tol), (b, r, h, float(np.max(err - tol)), float(err.max()))
                if len(at) == 0:
                    assert lse[b, r, h] == -math.inf and np.all(got[b, r, h] == 0)
                else:
                    bound = slack + ref.U32 * (4 * abs(wl) + len(at) + 16)
                    assert abs(lse[b, r, h] - wl) <= bound, (b, r, h, lse[b, r, h], wl)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(device, case):
    ctx, lead, n_max, nn, kind, Hq, Hkv, D, P, dtype, layout = ATTEND[case]
    say(f"[case] attention {case}: {ATTEND[case]}")
    k, v, table, seen, q = attention_problem(case)
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    got, lse = run_attention(device, ctx, lead, n_max, nn, seen, q, kv, case % 2)
    check_attention(ctx, lead, n_max, nn, seen, q, k, v, table, P, got, lse, D ** -0.5, dtype, case % 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kind", ["one", "tree", "chunk"])
def test_attention_missing_pages_and_odd_strides(device, dtype, kind):
    """Pages outside the pool and slots behind the table are unseen; rows of
    queries and outputs that are slices of wider ones; another scale."""
    say(f"[case] missing pages {dtype} {kind}")
    spec = dict(one=([90, 9], 1, 0, None, None, 8, 2, 128, 16, dtype, "slots"),
                tree=([70, 200], 1, 40, [40, 33], "tree", 8, 2, 128, 16, dtype, "slots"),
                chunk=([50, 128], 0, 140, [139, 140], None, 8, 2, 128, 16, dtype, "slots"))[kind]
    ctx, lead, n_max, nn, _, Hq, Hkv, D, P, _, _ = spec
    k, v, table, seen, q = attention_problem(50, spec=spec)
    table[0, 1], table[1, 0] = k.shape[1] + 5, -7
    table = np.ascontiguousarray(table[:, :max(2, table.shape[1] - 2)])
    wide = torch.randn(2, lead + n_max, Hq + 3, D).to(dtype)
    wide[:, :, :Hq] = q
    q = wide[:, :, :Hq]
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    got, lse = run_attention(device, ctx, lead, n_max, nn, seen, q, kv, 1, scale=0.25)
    check_attention(ctx, lead, n_max, nn, seen, q, k, v, table, P, got, lse, 0.25, dtype, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["tree", "chunk"])
def test_attention_unseen_values_stay_out(device, kind, D):
    """NaN and infinities in the keys and values of some tokens reach the rows
    that see them, and no other."""
    say(f"[case] unseen values {kind} {D}")
    ctx, lead, n_max, nn, Hq, Hkv, P, dtype = [70], 1 if kind == "tree" else 0, 80, [77], 4, 2, 16, BF16
    spec = (ctx, lead, n_max, nn, "tree" if kind == "tree" else None, Hq, Hkv, D, P, dtype, "slots")
    k, v, table, seen, q = attention_problem(60, spec=spec)
    clean_k, clean_v = k.clone(), v.clone()
    poison = {60: math.nan, 41: math.inf, 75: -math.inf}            # chunk rows
    for row, x in poison.items():
        at = ref.slot_at(table, k.shape[1], P, 0, ctx[0] + lead + row)
        v[1, at[0], at[1], 1, 5:D:7] = x
        if row != 41:
            k[1, at[0], at[1], 0] = math.nan
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    got, lse = run_attention(device, ctx, lead, n_max, nn, seen, q, kv, 1)
    live = lead + nn[0]
    touched = {r: [p for p in poison if ctx[0] + lead + p in
                   ref.visible(ctx[0], lead, r, nn[0], None if seen is None or r < lead else seen[0, r - lead])]
               for r in range(live)}
    clean = [r for r in range(live) if not touched[r]]
    assert clean and len(clean) < live
    check_attention(ctx, lead, n_max, nn, seen, q, clean_k, clean_v, table, P, got, lse, D ** -0.5, dtype, 1,
                    rows=clean)
    for r in range(live):
        if not touched[r]:
            continue
        for h in (2, 3):                                            # key head 1: values only
            sums = {math.copysign(math.inf, poison[p]) if math.isinf(poison[p]) else math.nan for p in touched[r]}
            want = sums.pop() if len(sums) == 1 else math.nan
            col = got[0, r, h, 5:D:7]
            assert np.all(np.isnan(col)) if math.isnan(want) else np.all(col == want), (r, h, want, col)
            assert np.all(np.isfinite(got[0, r, h, 0:5]))
        if any(p != 41 for p in touched[r]):
            assert np.all(np.isnan(got[0, r, 0])) and np.isnan(lse[0, r, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("size", [30.0, 3000.0])
def test_attention_large_scores(device, size):
    """Scores whose differences pass exp's range: the running maximum carries."""
    spec = ([300, 70], 1, 20, [20, 9], "tree", 8, 2, 128, 16, BF16, "slots")
    ctx, lead, n_max, nn, _, Hq, Hkv, D, P, dtype, _ = spec
    say(f"[case] large scores {size}")
    k, v, table, seen, q = attention_problem(70, spec=spec)
    q = (q.float() * size).to(dtype)
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    got, lse = run_attention(device, ctx, lead, n_max, nn, seen, q, kv, 0)
    check_attention(ctx, lead, n_max, nn, seen, q, k, v, table, P, got, lse, D ** -0.5, dtype, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("ragged", [False, True])
def test_attention_long_contexts(device, ragged):
    """Long contexts beside short ones, against fp64 on the GPU machine's CPU."""
    ctx = [20000, 3, 0, 517, 8191] if ragged else [30000]
    spec = (ctx, 1, 0, None, None, 8, 2, 128, 16, BF16, "slots")
    _, lead, n_max, nn, _, Hq, Hkv, D, P, dtype, _ = spec
    say(f"[case] long {ctx}")
    k, v, table, seen, q = attention_problem(80, spec=spec)
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    got, lse = run_attention(device, ctx, lead, n_max, nn, seen, q, kv, 1)
    check_attention(ctx, lead, n_max, nn, seen, q, k, v, table, P, got, lse, D ** -0.5, dtype, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["one", "few", "tree", "chunk"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_behind_a_wide_page_table(device, kind, D):
    """A page table for far longer contexts than there are: the split is
    derived from the lengths, and few segments go over resident workgroups."""
    say(f"[case] wide table {kind} {D}")
    spec = dict(one=([2900], 1, 0, None, None, 8, 2, D, 16, BF16, "slots"),
                few=([700, 1], 1, 15, [15, 9], "tree", 4, 1, D, 16, F16, "slots"),
                tree=([1500], 1, 64, [61], "tree", 4, 1, D, 8, BF16, "slots"),
                chunk=([300], 0, 200, [199], None, 4, 1, D, 24, F16, "slots"))[kind]
    ctx, lead, n_max, nn, _, Hq, Hkv, _, P, dtype, _ = spec
    k, v, table, seen, q = attention_problem(90, spec=spec)
    wide = np.full((len(ctx), 20000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(wide).to(device))
    got, lse = run_attention(device, ctx, lead, n_max, nn, seen, q, kv, 0)
    check_attention(ctx, lead, n_max, nn, seen, q, k, v, wide, P, got, lse, D ** -0.5, dtype, 0)


@pytest.mark.gpu
def test_attention_of_many_requests(device):
    """More requests than a wave has lanes, of very different lengths, some
    without rows, some without nodes; also more than the chunk search takes."""
    for B, ctx_of in ((150, lambda i: [-1, 0, 17, 900][i % 4] + i % 3), (700, lambda i: (i * 7) % 90)):
        say(f"[case] {B} requests")
        ctx = [max(ctx_of(i), -1) for i in range(B)]
        nn = [(i * 5) % 4 for i in range(B)]
        spec = (ctx, 1, 3, nn, "tree", 2, 1, 64, 16, BF16, "slots")
        k, v, table, seen, q = attention_problem(91, spec=spec)
        dk, dv = pair_on_device(k, v, device)
        kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
        got, lse = run_attention(device, ctx, 1, 3, nn, seen, q, kv, 0)
        check_attention(ctx, 1, 3, nn, seen, q, k, v, table, 16, got, lse, 0.125, BF16, 0)


@pytest.mark.gpu
def test_attention_of_the_largest_batch(device):
    """65535 requests of one token each: a row that sees one key is its value."""
    say("[case] largest batch")
    B, Hkv, D = 65535, 8, 64
    gen = torch.Generator(device=device).manual_seed(1)
    k, v = (torch.empty(B, 1, Hkv, D, dtype=BF16, device=device).normal_(generator=gen) for _ in range(2))
    table = torch.randperm(B, device=device).to(torch.int32)[:, None].contiguous()
    kv = bd.KVCache(k, v, table)
    chunk = bd.Chunk(torch.zeros(B, dtype=torch.int32, device=device))
    q = torch.empty(B, 1, Hkv, D, dtype=BF16, device=device).normal_(generator=gen)
    out = torch.zeros_like(q)
    ws = torch.empty(bd.dt_attention_workspace(kv, chunk, Hkv), dtype=torch.uint8, device=device)
    bd.dt_tree_attention(kv, chunk, q, out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 0], v[table[:, 0].long(), 0])


@pytest.mark.gpu
def test_lengths_beyond_the_table(device):
    """ctx_len up to the largest int32: slots behind the table are dropped on
    writing and unseen on reading."""
    say("[case] lengths beyond the table")
    P, D, far = 16, 64, 2 ** 31 - 1
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(3, P, 1, D, generator=gen).to(BF16).to(device) for _ in range(2))
    was = k.clone(), v.clone()
    table = torch.tensor([[2, 0, 1], [1, 2, 0]], dtype=torch.int32, device=device)
    kv = bd.KVCache(k, v, table)
    x = torch.randn(2, 5, 1, D, generator=gen).to(BF16).to(device)
    chunk = bd.Chunk(torch.tensor([far, far - 3], dtype=torch.int32, device=device), 5)
    freqs = bd.dt_rope_frequencies(D, 10000.0)[0].to(device)
    q = torch.empty_like(x)
    bd.dt_kv_append(kv, chunk, x, x, q=x, q_out=q, freqs=freqs)
    torch.cuda.synchronize()
    assert torch.equal(k, was[0]) and torch.equal(v, was[1])
    want, size = ref.append_head(x[0, 4, 0].cpu().double().numpy(), None, 0, far + 4, freqs.cpu().numpy(), False, 1.0)
    assert np.all(np.abs(q[0, 4, 0].cpu().double().numpy() - want) <= ref.append_tolerance(want, size, BF16))
    got, lse = run_attention(device, [far, far - 3], 5, 0, None, None, x.cpu(), kv, 0)
    host = table.cpu().numpy()
    for b in range(2):
        K, V = (torch.cat([t[p] for p in host[b]]).cpu().double().numpy()[:, 0] for t in (k, v))
        for r in range(5):
            w, _, spread, slack, vmax = ref.attend_row(x[b, r, 0].cpu().double().numpy(), K, V, D ** -0.5)
            assert np.all(np.abs(got[b, r, 0] - w) <= ref.attend_tolerance(w, spread, slack, vmax, 48, BF16))


@pytest.mark.parametrize("index,current,moved", [(-1, 0, []), (0, 0, []), (1, 0, [1]), (0, 1, [0])])
def test_calls_are_made_on_their_tensors_device(monkeypatch, index, current, moved):
    """A device's default stream has a null handle, so the call has to be made
    with that device current, and leaves the current one as it was."""
    seen = []

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            seen.append(self.i)

        def __exit__(self, *exc):
            seen.append("left")

    monkeypatch.setattr(bd, "_current_device", lambda: current)
    monkeypatch.setattr(torch.cuda, "device", Device)

    def call(x, y):
        assert seen == moved
        return x + y

    assert bd._on_device(index, call, 2, 3) == 5
    assert seen == (moved + ["left"] if moved else [])


def test_every_call_goes_through_its_device(monkeypatch):
    """The four entry points that launch are called by way of their tensors' device."""
    seen = []
    monkeypatch.setattr(bd, "_on_device", lambda index, call, *args: seen.append((index, call.__name__)) or 0)
    k = torch.zeros(2, 16, 1, 64, dtype=BF16)
    kv = bd.KVCache(k, torch.zeros_like(k), torch.zeros(1, 2, dtype=torch.int32))
    chunk = bd.Chunk(torch.zeros(1, dtype=torch.int32))
    x = torch.zeros(1, 1, 1, 64, dtype=BF16)
    i32 = torch.zeros(1, 1, dtype=torch.int32)
    bd.dt_kv_append(kv, chunk, x, x)
    bd.dt_tree_attention(kv, chunk, x, torch.empty_like(x))
    bd.dt_process_logits(torch.zeros(1, 1, 32), torch.zeros(1, 1, 32))
    bd.dt_commit_path(kv, chunk, None, None, i32, i32.clone(), torch.zeros(1, dtype=torch.int32))
    assert seen == [(-1, name) for name in ("dt_kv_append", "dt_tree_attention", "dt_process_logits",
                                            "dt_commit_path")]


@pytest.mark.gpu
def test_calls_in_flight_on_two_streams(device):
    """Appends, attention and logits of two batches on two streams, each with
    its own workspace, give each call's own results; so does a side stream
    passed to the call instead of the current one."""
    say("[case] two streams")
    jobs = []
    for i, spec in enumerate((([4000, 35, 812], 1, 20, [20, 7, 15], "tree", 8, 2, 128, 16, BF16, "slots"),
                              ([3000, 700], 1, 0, None, None, 8, 2, 128, 16, BF16, "slots"))):
        k, v, table, seen, q = attention_problem(95 + i, spec=spec)
        dk, dv = pair_on_device(k, v, device)
        kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
        i32 = dict(dtype=torch.int32, device=device)
        mask = None if seen is None else torch.from_numpy(ref.pack_bits(seen)).to(device)
        chunk = bd.Chunk(torch.tensor(spec[0], **i32), spec[1], spec[2],
                         None if spec[3] is None else torch.tensor(spec[3], **i32), mask=mask)
        ws = torch.empty(bd.dt_attention_workspace(kv, chunk, 8), dtype=torch.uint8, device=device)
        dq = to_device(q, device)
        x = torch.randn(4, 3, 20001, device=device)
        hist = torch.randint(0, 20001, (4, 500), **i32)
        hlen = torch.full((4,), 500, **i32)
        freq = torch.full((4,), 0.25, device=device)
        jobs.append((kv, chunk, dq, torch.zeros_like(dq), ws, x, torch.zeros_like(x), hist, hlen, freq,
                     torch.cuda.Stream()))

    def call(j, **kw):
        bd.dt_tree_attention(j[0], j[1], j[2], j[3], workspace=j[4], **kw)
        bd.dt_process_logits(j[5], j[6], history=j[7], history_len=j[8], frequency=j[9], **kw)

    alone = []
    for j in jobs:
        call(j)
        torch.cuda.synchronize()
        alone.append((j[3].clone(), j[6].clone()))
        j[3].zero_(), j[6].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            call(j, stream=j[10])
    torch.cuda.synchronize()
    for j, (o, y) in zip(jobs, alone):
        assert torch.equal(j[3], o) and torch.equal(j[6], y)


@pytest.mark.gpu
def test_cache_beyond_32_bit_offsets(device):
    """Pages more than 2^31 elements into the pool: append, attend, commit."""
    say("[case] 64-bit offsets")
    P, Hkv, D, step, pages = 16, 1, 64, 1 << 26, 40
    pool = torch.empty(pages * step + P * D * 2, dtype=BF16, device=device)
    shape, stride = (pages, P, Hkv, D), (step, D, D, 1)
    k, v = pool.as_strided(shape, stride), pool.as_strided(shape, stride, P * D)
    table = torch.tensor([[39, 2, 38]], dtype=torch.int32, device=device)
    kv = bd.KVCache(k, v, table)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(1, 40, 3, D, generator=gen).to(BF16)
    i32 = dict(dtype=torch.int32, device=device)
    zero = torch.zeros(1, **i32)
    dx = x.to(device)
    bd.dt_kv_append(kv, bd.Chunk(zero, 0, 40), dx[:, :, 1:2], dx[:, :, 2:3])
    torch.cuda.synchronize()
    flat = torch.cat([k[p] for p in (39, 2, 38)]).cpu()
    assert torch.equal(flat[:40], x[0, :, 1:2])
    q, out = dx[:, :, 0:1].contiguous(), torch.empty(1, 40, 1, D, dtype=BF16, device=device)
    chunk = bd.Chunk(zero, 0, 40)
    ws = torch.empty(max(bd.dt_attention_workspace(kv, chunk, 1), 16), dtype=torch.uint8, device=device)
    bd.dt_tree_attention(kv, chunk, q, out, workspace=ws)
    torch.cuda.synchronize()
    got = out.cpu().double().numpy()
    for r in range(40):
        want, _, spread, slack, vmax = ref.attend_row(x[0, r, 0].double().numpy(), x[0, :r + 1, 1].double().numpy(),
                                                      x[0, :r + 1, 2].double().numpy(), D ** -0.5)
        assert np.all(np.abs(got[0, r, 0] - want) <= ref.attend_tolerance(want, spread, slack, vmax, r + 1, BF16))
    tokens, parents = torch.tensor([[5, 6, 7]], **i32), torch.tensor([[-1, -1, 1]], **i32)
    target = torch.tensor([[6, 0, 7, 9]], **i32)
    accepted, lengths = torch.zeros(1, 4, **i32), torch.zeros(1, **i32)
    bd.dt_commit_path(kv, bd.Chunk(torch.tensor([36], **i32), 1, 3), tokens, parents, target, accepted, lengths)
    torch.cuda.synchronize()
    assert accepted.tolist() == [[6, 7, 9, -1]] and lengths.tolist() == [3]
    assert torch.equal(k[38, 5:7].cpu(), x[0, 38:40, 1:2]) and torch.equal(v[38, 5:7].cpu(), x[0, 38:40, 2:3])


# ---------------------------------------------------------------------------
# dt_process_logits
# ---------------------------------------------------------------------------

LOGITS = [
    # B, lead, n_max, n_nodes, V, dtype, history, n_bias, grammar, tree, in place
    (1, 1, 0, None, 1, F32, 4, 0, None, False, False),
    (1, 1, 0, None, 33, BF16, 0, 3, "rows", False, False),
    (2, 3, 0, None, 1000, F32, 50, 0, None, False, True),
    (3, 1, 9, [9, 0, 4], 5001, BF16, 300, 20, "index", True, False),
    (2, 2, 40, [40, 33], 4099, F32, 1000, 300, "index", True, True),
    (2, 8, 0, None, 32000, BF16, 5000, 64, "index", False, False),
    (1, 1, 64, [61], 32000, F32, 700, 16, None, True, False),
    (1, 4, 0, None, 151936, BF16, 2000, 10, "rows", False, True),
    (2, 0, 5, [5, 3], 12289, BF16, 0, 0, "rows", True, False),
    (1, 2, 0, None, 8195, BF16, 100000, 0, None, False, False),
    (2, 3, 0, None, 8191, BF16, 0, 0, None, False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(LOGITS)))
def test_logits(device, case):
    B, lead, n_max, nn, V, dtype, H, nb, grammar, tree, inplace = LOGITS[case]
    say(f"[case] logits {case}: {LOGITS[case]}")
    rs = np.random.RandomState(300 + case)
    rows, words = lead + n_max, (V + 31) // 32
    x = torch.from_numpy((3 * rs.randn(B, rows, V)).astype(np.float32)).to(dtype)
    x[rs.rand(B, rows, V) < 0.05] = -math.inf
    x[rs.rand(B, rows, V) < 0.02] = 0.0
    hist = (V * rs.rand(B, H) ** 3).astype(np.int32)
    hist[rs.rand(B, H) < 0.02] = V
    hist[rs.rand(B, H) < 0.02] = -1
    hlen = np.array([H + 3, H // 2, 0][:B], np.int32)
    plen = np.array([H // 4, H + 9, -2][:B], np.int32)
    rep, freq, pres = (rs.uniform(lo, hi, B).astype(np.float32) for lo, hi in ((0.8, 1.6), (-0.2, 0.5), (0, 1)))
    ids = (V * rs.rand(B, nb) ** 2).astype(np.int32)
    ids[:, nb // 2:nb // 2 + 2] = -1
    bias = rs.uniform(-4, 4, (B, nb)).astype(np.float32)
    bias[rs.rand(B, nb) < 0.1] = -math.inf
    tokens = (V * rs.rand(B, n_max) ** 3).astype(np.int32)
    clamped = nn or [n_max] * B
    seen = ref.random_tree(rs, B, n_max, clamped)[2] if tree else None
    if tree and n_max > 8:
        seen[:, 2, 5:] = True                                  # any bits, also behind n_nodes
    states = 5 if grammar == "index" else B * rows
    ok = rs.rand(states, V) < rs.choice([0.02, 0.5, 0.98, 1.0, 0.0], (states, 1))
    index = rs.randint(-2, states + 2, (B, rows)).astype(np.int32) if grammar == "index" else None
    d = lambda a: to_device(a, device)                         # noqa: E731
    dx = d(x)
    out = dx if inplace else torch.full_like(dx, SENTINEL)
    bd.dt_process_logits(dx, out, history=d(hist) if H else None, history_len=d(hlen), prompt_len=d(plen),
                         repetition=d(rep), frequency=d(freq), presence=d(pres), bias_ids=d(ids) if nb else None,
                         bias=d(bias) if nb else None, allow=d(ref.pack_bits(ok)) if grammar else None,
                         allow_index=d(index), lead=lead, n_nodes=None if nn is None else d(np.array(nn, np.int32)),
                         node_tokens=d(tokens) if tree else None,
                         node_mask=d(ref.pack_bits(seen)) if tree else None)
    torch.cuda.synchronize()
    got = out.cpu()
    bits = torch.int16 if dtype == BF16 else torch.int32
    for b in range(B):
        n = min(max(int(hlen[b]), 0), H)
        p = min(max(int(plen[b]), 0), n)
        inside = lambda a: a[(a >= 0) & (a < V)]               # noqa: E731
        base = np.bincount(inside(hist[b, p:n]), minlength=V)
        prompt = np.bincount(inside(hist[b, :p]), minlength=V) > 0
        add = np.zeros(V)
        for i, t in zip(ids[b], bias[b]):
            if 0 <= i < V:
                add[i] = t
        live = lead + clamped[b]
        rest = x[b, live:] if inplace else torch.full_like(x[b, live:], SENTINEL)
        assert torch.equal(got[b, live:], rest)
        for r in range(live):
            count = base
            if tree and r >= lead:
                count = base + np.bincount(inside(tokens[b, :clamped[b]][seen[b, r - lead, :clamped[b]]]),
                                           minlength=V)
            allowed = None
            if grammar:
                i = b * rows + r if index is None else int(index[b, r])
                allowed = ok[i] if 0 <= i < states else None
            want, size, touched = ref.logits_row(x[b, r].float().numpy(), count, prompt, float(rep[b]),
                                                 float(freq[b]), float(pres[b]), add, allowed)
            have = got[b, r].double().numpy()
            low = np.isneginf(want)
            assert np.array_equal(np.isneginf(have), low), (b, r)
            # six fp32 operations, each half a step of the largest value in reach; then the result's own
            tol = ref.HALF_STEP[dtype] * np.abs(want) + 6 * ref.U32 * size + ref.SMALLEST[dtype]
            bad = ~low & ~(np.abs(have - np.where(low, 0, want)) <= np.where(low, 0, tol))
            assert not bad.any(), (b, r, np.flatnonzero(bad)[:5])
            same = torch.from_numpy(~touched & ~low)
            assert torch.equal(got[b, r][same].view(bits), x[b, r][same].view(bits))


@pytest.mark.gpu
def test_logits_nan_in_masked_places_and_neutral_call(device):
    say("[case] logits nan")
    V = 1003
    x = torch.randn(1, 2, V)
    x[0, 0, 5:900:3] = math.nan
    x[0, 0, 6:900:3] = math.inf
    ok = np.ones((2, V), bool)
    ok[0, 5:900:3] = ok[0, 6:900:3] = False
    for dtype in (F32, BF16):
        dx = x.to(dtype).to(device)
        out = torch.empty_like(dx)
        bd.dt_process_logits(dx, out, allow=to_device(ref.pack_bits(ok), device))
        torch.cuda.synchronize()
        want = x.to(dtype).clone()
        want[torch.from_numpy(~ok)[None]] = -math.inf
        assert torch.equal(out.cpu(), want)
        bd.dt_process_logits(dx, out)
        torch.cuda.synchronize()
        bits = torch.int16 if dtype == BF16 else torch.int32
        assert torch.equal(out.cpu().view(bits), x.to(dtype).view(bits))


# ---------------------------------------------------------------------------
# dt_commit_path
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("case", range(8))
def test_commit(device, case):
    rs = np.random.RandomState(40 + case)
    B = [1, 5, 3, 2, 4, 70, 2, 3][case]
    n_max = [0, 12, 64, 200, 1024, 33, 7, 64][case]
    lead = [1, 1, 2, 3, 1, 1, 1, 1][case]
    L = [3, 13, 65, 4, 1025, 20, 1, 9][case]
    width = [4, 3, 4, 1, 1, 4, 2, 8][case]                     # width 1: one path as deep as the tree
    Hkv, D, P = [(1, 64, 16), (2, 128, 8), (8, 128, 16), (1, 256, 1), (1, 64, 64), (1, 64, 16), (3, 64, 24),
                 (4, 128, 32)][case]
    dtype, layers, layout = [BF16, F16][case % 2], [1, 3, 2, 5, 1, 1, 2, 4][case], ["slots", "heads", "both"][case % 3]
    say(f"[case] commit {case}: B {B} n_max {n_max} lead {lead} L {L}")
    nn = [int(rs.randint(0, n_max + 1)) if i else n_max for i in range(B)]
    ctx = [int(c) for c in rs.randint(0, 60, B)]
    if B > 2:
        ctx[1] = -1
    k, v, table = make_cache(rs, ctx, lead + n_max, P, Hkv, D, dtype, layers=layers, layout=layout)
    k, v = torch.nan_to_num(k, nan=1.5), torch.nan_to_num(v, nan=-2.5)
    k[:], v[:] = torch.randn(k.shape).to(dtype), torch.randn(v.shape).to(dtype)
    if case == 7:
        table[2, (ctx[2] + lead + 9) // P] = -1                # a source page that does not exist
    parents = ref.random_tree(rs, B, n_max, nn, width=width)[0]
    tokens = rs.randint(0, 4, (B, n_max)).astype(np.int32)     # few tokens: siblings repeat, paths get long
    target = rs.randint(0, 4, (B, lead + n_max)).astype(np.int32)
    if width == 1:
        for b in range(B):
            target[b, lead - 1:lead - 1 + n_max] = tokens[b]
    if n_max > 20:
        parents[0, 15] = 15                                    # malformed: its own parent
    i32 = dict(dtype=torch.int32, device=device)
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    chunk = bd.Chunk(torch.tensor(ctx, **i32), lead, n_max, torch.tensor(nn, **i32))
    accepted, nodes = (torch.full((B, L), 99, **i32) for _ in range(2))
    lengths = torch.full((B,), 99, **i32)
    bd.dt_commit_path(kv, chunk, to_device(tokens, device), to_device(parents, device), to_device(target, device),
                      accepted, lengths, nodes=nodes)
    torch.cuda.synchronize()
    for b in range(B):
        said, path = ([], []) if ctx[b] < 0 else ref.walk(tokens[b], parents[b], target[b], lead, nn[b], L)
        assert accepted[b].tolist() == said + [-1] * (L - len(said))
        assert nodes[b].tolist() == path + [-1] * (L - len(path))
        assert int(lengths[b]) == len(said)
        at = lambda i: ref.slot_at(table, k.shape[1], P, b, ctx[b] + lead + i)   # noqa: E731
        for cache in (k, v):
            old = [None if at(n) is None else cache[:, at(n)[0], at(n)[1]].clone() for n in path]
            for i, x in enumerate(old):
                if x is not None and at(i) is not None:
                    cache[:, at(i)[0], at(i)[1]] = x
    assert torch.equal(dk.cpu(), k) and torch.equal(dv.cpu(), v)
    again, len2 = torch.zeros(B, L, **i32), torch.zeros(B, **i32)
    bd.dt_commit_path(None, chunk, to_device(tokens, device), to_device(parents, device), to_device(target, device),
                      again, len2)                             # tokens only
    assert torch.equal(again, accepted) and torch.equal(len2, lengths)
    assert torch.equal(dk.cpu(), k)


# ---------------------------------------------------------------------------
# the pass as a whole
# ---------------------------------------------------------------------------

def _step(bd, dp, kv, chunk, x, freqs, q_out, o, ws, head, hist, hist_len, logits, top, accepted, lengths, Hq, Hkv):
    """One verification round: build, append, attend, head, penalties, choice, commit, table update."""
    bd.dt_build_tree(dp.logits, dp.ngram, dp.params, dp.out)
    bd.dt_kv_append(kv, chunk, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], q=x[:, :, :Hq], q_out=q_out, freqs=freqs)
    bd.dt_tree_attention(kv, chunk, q_out, o, workspace=ws)
    torch.mm(o.flatten(0, 1).flatten(1, 2), head, out=logits.view(-1, logits.shape[-1]))
    top["ids"].copy_(dp.out.tokens[:, 1:2])      # a bias that makes the target choose node 1's token everywhere
    bd.dt_process_logits(logits, logits, history=hist, history_len=hist_len, frequency=top["freq"], lead=chunk.lead,
                         bias_ids=top["ids"], bias=top["bias"], n_nodes=dp.out.n_nodes, node_tokens=dp.out.tokens,
                         node_mask=dp.out.mask)
    bd.dt_position_topk(logits, top["params"], top["lse"], top["tok"], top["val"])
    bd.dt_commit_path(kv, chunk, dp.out.tokens, dp.out.parents, top["tok"].view(chunk.B, chunk.rows), accepted,
                      lengths)
    bd.dt_ngram_update(dp.ngram, dp.params.ctx, accepted, lengths)


@pytest.mark.gpu
def test_round_as_it_is_used_and_captured(device):
    """Built trees through the whole pass: each operator's outputs against the
    64-bit definitions, then the same round captured into a graph, replayed
    with eager work between, equal to the eager result each time."""
    say("[case] round")
    p = synth.make_problem("c4Lp", 3, B=3, hash_cap_log2=12, hash_keys_log2=10)
    dp = bd.upload_problem(p, device, budget=31)
    B, budget, lead, Hq, Hkv, D, P, V = 3, 31, 1, 4, 2, 64, 16, p.V
    rs = np.random.RandomState(1)
    ctx = [20, 77, 5]
    k, v, table = make_cache(rs, ctx, lead + budget, P, Hkv, D, BF16)
    dk, dv = pair_on_device(k, v, device)
    kv = bd.KVCache(dk, dv, torch.from_numpy(table).to(device))
    i32 = dict(dtype=torch.int32, device=device)
    chunk = bd.Chunk.of_tree(torch.tensor(ctx, **i32), dp.out, lead)
    x = torch.from_numpy(rs.randn(B, lead + budget, Hq + 2 * Hkv, D).astype(np.float32)).to(BF16).to(device)
    freqs = bd.dt_rope_frequencies(D, 10000.0)[0].to(device)
    q_out = torch.zeros(B, lead + budget, Hq, D, dtype=BF16, device=device)
    o = torch.zeros_like(q_out)
    ws = torch.empty(max(bd.dt_attention_workspace(kv, chunk, Hq), 16), dtype=torch.uint8, device=device)
    head = torch.from_numpy(rs.randn(Hq * D, V).astype(np.float32)).to(BF16).to(device)
    hist = torch.from_numpy(rs.randint(0, V, (B, 40)).astype(np.int32)).to(device)
    hist_len = torch.tensor([40, 11, 0], **i32)
    logits = torch.zeros(B, chunk.rows, V, dtype=BF16, device=device)
    R = B * chunk.rows
    tp = bd.Params(B=R, V=V, d=1, k=1, W=1, budget=1, dtype=bd.DT_DTYPE_BF16)
    tp.workspace = torch.empty(bd.dt_workspace_size(tp), dtype=torch.uint8, device=device)
    top = dict(params=tp, lse=torch.empty(R, dtype=torch.float64, device=device),
               tok=torch.empty(R, 1, **i32), val=torch.empty(R, 1, device=device),
               freq=torch.tensor([0.5, 0.0, 0.1], device=device), ids=torch.zeros(B, 1, **i32),
               bias=torch.full((B, 1), 1000.0, device=device))
    accepted, lengths = torch.zeros(B, 9, **i32), torch.zeros(B, **i32)
    bd.dt_build_tree(dp.logits, dp.ngram, dp.params, dp.out)
    torch.cuda.synchronize()
    args = (bd, dp, kv, chunk, x, freqs, q_out, o, ws, head, hist, hist_len, logits, top, accepted, lengths, Hq, Hkv)
    start = (dk.clone(), dv.clone(), dp.ngram.keys.clone(), dp.ngram.succ.clone())

    def reset():
        for t, s in zip((dk, dv, dp.ngram.keys, dp.ngram.succ), start):
            t.copy_(s)
        for t in (q_out, o, logits, accepted, lengths):
            t.zero_()

    reset()
    _step(*args)
    torch.cuda.synchronize()
    tree = dp.out.numpy()
    nn = tree["n_nodes"].tolist()
    assert min(nn) > 5
    seen = np.unpackbits(tree["mask"].view(np.uint8), axis=-1, bitorder="little")[..., :budget].astype(bool)
    xs = x.cpu().double().numpy()
    for b in range(B):
        for r in range(lead + nn[b]):
            pos = ctx[b] + r if r < lead else ctx[b] + lead - 1 + int(tree["depths"][b, r - lead])
            for h in range(Hq):
                want, size = ref.append_head(xs[b, r, h], None, 0, pos, freqs.cpu().numpy(), False, 1.0)
                have = q_out[b, r, h].cpu().double().numpy()
                assert np.all(np.abs(have - want) <= ref.append_tolerance(want, size, BF16))
    host = dk.cpu(), dv.cpu()
    said = top["tok"].view(B, -1).cpu().numpy()
    got = o.cpu().double().numpy()
    taken, count = accepted.tolist(), lengths.tolist()
    reset()
    bd.dt_build_tree(dp.logits, dp.ngram, dp.params, dp.out)
    bd.dt_kv_append(kv, chunk, x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], q=x[:, :, :Hq], q_out=q_out, freqs=freqs)
    torch.cuda.synchronize()
    lse = np.full((B, chunk.rows, Hq), SENTINEL)
    mk, mv = dk.cpu(), dv.cpu()
    for b in range(B):
        for r in range(lead + nn[b]):
            slots = ref.visible(ctx[b], lead, r, nn[b], None if r < lead else seen[b, r - lead])
            at = [ref.slot_at(table, k.shape[1], P, b, s) for s in slots]
            pg, off = (torch.tensor([a[i] for a in at], dtype=torch.long) for i in (0, 1))
            K, Vv = mk[0, pg, off].double().numpy(), mv[0, pg, off].double().numpy()
            for h in range(Hq):
                want, _, spread, slack, vmax = ref.attend_row(q_out[b, r, h].cpu().double().numpy(), K[:, h // 2],
                                                              Vv[:, h // 2], D ** -0.5)
                tol = ref.attend_tolerance(want, spread, slack, vmax, len(at), BF16)
                assert np.all(np.abs(got[b, r, h] - want) <= tol), (b, r, h)
    for b in range(B):
        words, path = ref.walk(tree["tokens"][b], tree["parents"][b], said[b], lead, nn[b], 9)
        assert taken[b] == words + [-1] * (9 - len(words)) and count[b] == len(words)
        assert path[0] == 1 and int(said[b, 0]) == int(tree["tokens"][b, 1])
        for i, n in enumerate(path):
            src = ref.slot_at(table, k.shape[1], P, b, ctx[b] + lead + n)
            dst = ref.slot_at(table, k.shape[1], P, b, ctx[b] + lead + i)
            assert torch.equal(host[0][0, dst[0], dst[1]], mk[0, src[0], src[1]])
            assert torch.equal(host[1][0, dst[0], dst[1]], mv[0, src[0], src[1]])
    # eager results to compare replays with
    reset()
    _step(*args)
    torch.cuda.synchronize()
    result = [t.clone() for t in (dk, dv, q_out, o, logits, accepted, lengths)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        reset()
        _step(*args)
    torch.cuda.synchronize()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(*args)
    for i in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        bits = lambda t: t.view(torch.int16) if t.dtype == BF16 else t       # noqa: E731
        for a, w in zip((dk, dv, q_out, o, logits, accepted, lengths), result):
            assert torch.equal(bits(a), bits(w)), f"replay {i}"
        torch.randn(1000, 1000, device=device).mm(torch.randn(1000, 1000, device=device))
