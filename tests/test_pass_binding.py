"""What the Python entry points of the verification pass refuse before anything
is launched (no GPU needed)."""

import pytest
import torch

bd = pytest.importorskip("draft_tree_construction_dt_amd.binding")

I32 = torch.int32


def _calls(B):
    """The four launching entry points on host tensors, for a batch of B."""
    k = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    kv = bd.KVCache(k, torch.zeros_like(k), torch.zeros(max(B, 1), 2, dtype=I32))
    chunk = bd.Chunk(torch.zeros(B, dtype=I32))
    x = torch.zeros(B, 1, 1, 64, dtype=torch.bfloat16)
    ws = torch.empty(max(bd.dt_attention_workspace(kv, chunk, 1), 16), dtype=torch.uint8)
    choice, out, n = torch.zeros(B, 1, dtype=I32), torch.zeros(B, 1, dtype=I32), torch.zeros(B, dtype=I32)
    return {
        "dt_kv_append": lambda: bd.dt_kv_append(kv, chunk, x, x),
        "dt_tree_attention": lambda: bd.dt_tree_attention(kv, chunk, x, torch.empty_like(x), workspace=ws),
        "dt_process_logits": lambda: bd.dt_process_logits(torch.zeros(B, 1, 32), torch.zeros(B, 1, 32)),
        "dt_commit_path": lambda: bd.dt_commit_path(kv, chunk, None, None, choice, out, n),
        "dt_commit_path, tokens only": lambda: bd.dt_commit_path(None, chunk, None, None, choice, out, n),
    }


@pytest.mark.parametrize("name", list(_calls(1)))
def test_host_tensors_are_refused(monkeypatch, name):
    """Tensors that are all in host memory agree about their device, and no
    kernel may be given their addresses.  Nothing is called in the library."""
    reached = []
    real = bd._load()

    class Library:
        def __getattr__(self, fn):
            if fn == "dt_status_string":
                return real.dt_status_string

            def call(*args):
                reached.append(fn)
                return bd.DT_OK
            call.__name__ = fn
            return call

    call = _calls(2)[name]
    monkeypatch.setattr(bd, "_load", lambda: Library())
    with pytest.raises(bd.DtError) as e:
        call()
    assert e.value.status == bd.DT_ERR_INVALID_ARG and name.split(",")[0] in str(e.value)
    assert not reached
    monkeypatch.setattr(bd, "_load", lambda: real)
    _calls(0)[name]()                                             # an empty batch launches nothing and is fine
