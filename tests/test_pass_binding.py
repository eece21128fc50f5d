"""What the Python entry points of the verification pass refuse before anything
is launched (no GPU needed)."""

import ctypes
from types import SimpleNamespace

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


@pytest.mark.parametrize("axis", ["layer_stride", "page_stride", "slot_stride", "head_stride"])
@pytest.mark.parametrize("stride", [0, 8, 120])
def test_caches_that_share_elements_are_read_only(axis, stride):
    """Heads, slots, pages or layers that overlap cannot be written: two
    workgroups would move the same element.  A batch of no requests launches
    nothing, so that the read is seen to be accepted."""
    fake, lib = 0x100000, bd._load()
    kv = bd._KVCache(k=fake, v=fake, page_table=fake, layer_stride=1 << 20, page_stride=16384, slot_stride=1024,
                     head_stride=128, layers=2, num_pages=9, page_size=16, max_pages=8, Hkv=8, D=128,
                     dtype=bd.DT_DTYPE_BF16)
    chunk = bd._Chunk(B=0, lead=1, n_max=8)
    append = bd._AppendParams(k=fake, v=fake, k_stride=1024, v_stride=1024, eps=1e-6, rot_scale=1.0)
    attend = bd._AttentionParams(q=fake, out=2 * fake, q_stride=4096, out_stride=4096, Hq=32, scale=0.1,
                                 workspace=fake, workspace_bytes=1 << 40)
    commit = bd._CommitParams(tokens=fake, parents=fake, target=fake, L=9, accepted=fake, lengths=fake)
    of = lambda p: (ctypes.byref(kv), ctypes.byref(chunk), ctypes.byref(p))      # noqa: E731
    assert lib.dt_kv_append(*of(append)) == lib.dt_commit_path(*of(commit)) == bd.DT_OK
    setattr(kv, axis, stride)
    assert lib.dt_kv_append(*of(append)) == lib.dt_commit_path(*of(commit)) == bd.DT_ERR_INVALID_ARG
    assert lib.dt_tree_attention(*of(attend)) == bd.DT_OK
    kv.layers = kv.num_pages = kv.page_size = kv.Hkv = 1           # strides of axes of length one are not read
    assert lib.dt_kv_append(*of(append)) == lib.dt_commit_path(*of(commit)) == bd.DT_OK


def test_streams_of_another_device_are_refused():
    """The library launches on its stream's device, which another device's
    tensors need not be mapped on."""
    stream = SimpleNamespace(cuda_stream=0x1230, device_index=1)
    assert bd._stream_of(stream, 1) == 0x1230 and bd._stream_of(0x77, 0) == 0x77
    with pytest.raises(bd.DtError) as e:
        bd._stream_of(stream, 0)
    assert e.value.status == bd.DT_ERR_INVALID_ARG
