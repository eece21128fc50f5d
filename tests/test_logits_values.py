"""dt_process_logits: single steps whose fp32 result is known to the bit, and
more biases than a chunk of the vocabulary has tokens."""

import numpy as np
import pytest
import torch

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("generated", [False, True])
@pytest.mark.parametrize("dense", [False, True])
def test_repetition_divides(device, generated, dense):
    """x / repetition is one fp32 division, also where 1 / repetition has no
    fp32 value or not all of its bits."""
    print("[case] repetition", generated, dense, flush=True)
    V = 9001
    rep = np.array([1.3, 0.7, 3.0, 1.1, 3e38, 1e-39, 2.0 ** -127, 2.0 ** -149, 1.0, 1.0000001], np.float32)
    B = len(rep)
    rs = np.random.RandomState(3)
    x = (rs.randn(B, 1, V) * 10.0 ** rs.uniform(-30, 4, (B, 1, V))).astype(np.float32)
    # runs of neighbours (a vector's tokens are then done all at once) or single tokens
    ids = np.tile(np.arange(0, V, 1 if dense else 5, dtype=np.int32), (B, 1))
    d = lambda a: torch.from_numpy(a).to(device)                 # noqa: E731
    n = d(np.full(B, ids.shape[1], np.int32))
    out = torch.empty(B, 1, V, device=device)
    bd.dt_process_logits(d(x), out, history=d(ids), history_len=n, prompt_len=None if generated else n,
                         repetition=d(rep))
    torch.cuda.synchronize()
    want = x.copy()
    with np.errstate(over="ignore", under="ignore"):
        y = np.where(x > 0, x / rep[:, None, None], x * rep[:, None, None])
    assert y.dtype == np.float32
    want[:, :, ids[0]] = y[:, :, ids[0]]
    assert np.array_equal(out.cpu().numpy().view(np.int32), want.view(np.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("n_bias,spread", [(5000, 4096), (65534, 9000), (4097, 1)])
def test_more_biases_than_a_chunk_has_tokens(device, n_bias, spread):
    """Ids drawn from few tokens: many are listed more than once in one chunk of
    4096, whose biases fill their table; the last entry of a token counts."""
    print("[case] biases", n_bias, spread, flush=True)
    B, rows, V = 3, 2, 9003
    rs = np.random.RandomState(n_bias)
    x = rs.randn(B, rows, V).astype(np.float32)
    ids = rs.randint(-1, spread, (B, n_bias)).astype(np.int32)
    bias = rs.uniform(-4, 4, (B, n_bias)).astype(np.float32)
    d = lambda a: torch.from_numpy(a).to(device)                 # noqa: E731
    for dtype in (F32, BF16):
        dx = d(x).to(dtype)
        out = torch.empty_like(dx)
        bd.dt_process_logits(dx, out, bias_ids=d(ids), bias=d(bias))
        torch.cuda.synchronize()
        for b in range(B):
            add = np.zeros(V, np.float32)
            for i, t in zip(ids[b], bias[b]):
                if i >= 0:
                    add[i] = t
            want = torch.from_numpy(dx[b].float().cpu().numpy() + add).to(dtype)     # one fp32 sum, rounded once
            assert torch.equal(out[b].cpu(), want)
