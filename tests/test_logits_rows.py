"""dt_process_logits where a workgroup takes several rows of a request one after
the other: a chunk of 4096 tokens of a request is shared by
ceil(2048 / (chunks * B)) workgroups, fewer than rows in every case here.
Against the definition in 64 bits (pass_ref.py), on a sample of the requests."""

import math

import numpy as np
import pytest
import torch

import pass_ref as ref

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

BF16, F32 = torch.bfloat16, torch.float32
SENTINEL = 7.0
I32 = torch.int32

CASES = {
    # B, lead, n_max, V, dtype, history, n_bias, grammar states, tree, in place, highest token of history and nodes
    "trees, 17 rows a workgroup": (64, 1, 64, 32000, F32, 700, 16, 0, True, False, 32000),
    "trees, the largest vocabulary": (64, 1, 12, 151936, BF16, 900, 64, 6, True, False, 151936),
    "three leading rows, 160 nodes in one chunk": (1024, 3, 160, 4099, BF16, 50, 0, 5, True, True, 600),
    "five leading rows of eleven": (700, 5, 6, 8200, F32, 300, 4, 0, True, True, 40),
    "70 rows without a tree": (1024, 70, 0, 4101, BF16, 80, 3, 7, False, True, 4101),
    "trees without leading rows": (300, 0, 90, 12289, F32, 0, 0, 4, True, False, 200),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_several_rows_a_workgroup(device, name):
    B, lead, n_max, V, dtype, H, nb, states, tree, inplace, top = CASES[name]
    print("[case]", name, flush=True)
    rows, chunks = lead + n_max, -(-V // 4096)
    assert -(-2048 // (chunks * B)) < rows                       # several rows a workgroup
    rs = np.random.RandomState(len(name))
    gen = torch.Generator(device=device).manual_seed(len(name))
    d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)   # noqa: E731
    x = torch.empty(B, rows, V, dtype=F32, device=device).normal_(generator=gen).mul_(3).to(dtype)
    hist = rs.randint(0, top, (B, H)).astype(np.int32)
    hlen, plen = rs.randint(0, H + 1, B).astype(np.int32), rs.randint(0, H // 2 + 1, B).astype(np.int32)
    rep, freq, pres = (rs.uniform(lo, hi, B).astype(np.float32) for lo, hi in ((0.8, 1.6), (0.2, 0.5), (0.5, 1)))
    ids = rs.randint(0, top, (B, nb)).astype(np.int32)
    bias = rs.uniform(-4, 4, (B, nb)).astype(np.float32)
    nn = rs.randint(n_max // 2, n_max + 1, B).astype(np.int32)
    tokens = rs.randint(0, top, (B, n_max)).astype(np.int32)
    seen = (rs.rand(B, n_max, n_max) < 0.5) if tree else None    # any bits, long overlapping paths
    ok = rs.rand(states, V) < 0.7
    index = rs.randint(-1, states + 1, (B, rows)).astype(np.int32)
    # of the sample every row, of the other requests the leading rows and the first of the tree
    whole = sorted({0, B - 1, B // 2, int(np.argmax(nn))})
    few = sorted(set(rs.choice(B, 24, replace=False).tolist()) - set(whole))
    was = {b: x[b].cpu() for b in whole + few}
    out = x if inplace else torch.full_like(x, SENTINEL)
    bd.dt_process_logits(x, out, history=d(hist) if H else None, history_len=d(hlen), prompt_len=d(plen),
                         repetition=d(rep), frequency=d(freq), presence=d(pres), bias_ids=d(ids) if nb else None,
                         bias=d(bias) if nb else None, allow=d(ref.pack_bits(ok)) if states else None,
                         allow_index=d(index) if states else None, lead=lead, n_nodes=d(nn),
                         node_tokens=d(tokens) if tree else None, node_mask=d(ref.pack_bits(seen)) if tree else None)
    torch.cuda.synchronize()
    bits = torch.int16 if dtype == BF16 else torch.int32
    for b in whole + few:
        got, n = out[b].cpu(), int(hlen[b])
        p = min(int(plen[b]), n)
        base = np.bincount(hist[b, p:n], minlength=V)
        prompt = np.bincount(hist[b, :p], minlength=V) > 0
        add = np.zeros(V)
        for i, t in zip(ids[b], bias[b]):
            add[i] = t
        live = lead + int(nn[b])
        assert torch.equal(got[live:], was[b][live:] if inplace else torch.full_like(was[b][live:], SENTINEL))
        for r in range(live) if b in whole else range(min(live, lead + 2)):
            count = base
            if tree and r >= lead:
                count = base + np.bincount(tokens[b, :nn[b]][seen[b, r - lead, :nn[b]]], minlength=V)
            allowed = ok[index[b, r]] if states and 0 <= index[b, r] < states else None
            want, size, touched = ref.logits_row(was[b][r].float().numpy(), count, prompt, float(rep[b]),
                                                 float(freq[b]), float(pres[b]), add, allowed)
            have, low = got[r].double().numpy(), np.isneginf(want)
            assert np.array_equal(np.isneginf(have), low), (b, r)
            # six fp32 operations, each half a step of the largest value in reach; then the result's own
            tol = ref.HALF_STEP[dtype] * np.abs(want) + 6 * ref.U32 * size + ref.SMALLEST[dtype]
            bad = ~low & ~(np.abs(have - np.where(low, 0, want)) <= np.where(low, 0, tol))
            assert not bad.any(), (b, r, np.flatnonzero(bad)[:5])
            same = torch.from_numpy(~touched & ~low)
            assert torch.equal(got[r][same].view(bits), was[b][r][same].view(bits))
