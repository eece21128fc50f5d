"""Python binding of libdt.so (include/dt.h): argument marshalling only.

Every step of the path runs in the library's HIP kernels.  torch supplies
device memory, the stream and (optionally) the profiling events; the
functions below only turn tensors into the plain pointers and sizes the C
ABI takes.  If the library is missing the import fails loudly: there is no
CPU fallback.
"""

from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass, field
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdt.so")

DT_OK, DT_ERR_INVALID_ARG, DT_ERR_UNSUPPORTED, DT_ERR_WORKSPACE, DT_ERR_HIP = 0, 1, 2, 3, 4
DT_DTYPE_F32, DT_DTYPE_BF16, DT_DTYPE_F16 = 0, 1, 2
DT_MODE_DART, DT_MODE_DARTREE, DT_MODE_DARTREE_FULL = 0, 1, 2
DT_NGRAM_NONE, DT_NGRAM_DENSE_BIGRAM, DT_NGRAM_CSR_BIGRAM, DT_NGRAM_HASH_TRIGRAM = 0, 1, 2, 3
DT_ROPE_NONE, DT_ROPE_LINEAR, DT_ROPE_WAVELENGTH, DT_ROPE_YARN = 0, 1, 2, 3


class DtError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dt_status_string(status)}")


class _NGram(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("min_logp", ctypes.c_float),
        ("dense_logp", ctypes.c_void_p),
        ("row_ptr", ctypes.c_void_p),
        ("col", ctypes.c_void_p),
        ("csr_logp", ctypes.c_void_p),
        ("nnz", ctypes.c_int64),
        ("keys", ctypes.c_void_p),
        ("succ", ctypes.c_void_p),
        ("hash_logp", ctypes.c_void_p),
        ("cap", ctypes.c_int64),
        ("S", ctypes.c_int32),
    ]


class _Params(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("V", ctypes.c_int32), ("d", ctypes.c_int32), ("k", ctypes.c_int32),
        ("W", ctypes.c_int32), ("budget", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("mode", ctypes.c_int32), ("ctx", ctypes.c_void_p), ("E", ctypes.c_void_p),
        ("F", ctypes.c_void_p), ("R", ctypes.c_int32), ("sweep_chunks", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p), ("prof_event_start", ctypes.c_void_p),
        ("prof_event_stop", ctypes.c_void_p),
    ]


def _fields(spec):
    kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "l": ctypes.c_int64, "f": ctypes.c_float,
             "z": ctypes.c_size_t}
    return [(name, kinds[kind]) for kind, names in spec for name in names.split()]


def _packer(struct_type):
    """The same structure as bytes from its fields' values, in a third of the
    time (a call of a few microseconds is made for every layer and token)."""
    kinds = {ctypes.c_void_p: "P", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f",
             ctypes.c_size_t: "N"}
    packer = struct.Struct("@" + "".join(kinds[kind] for _, kind in struct_type._fields_) + "0q")
    assert packer.size == ctypes.sizeof(struct_type)
    return packer.pack


class _KVCache(ctypes.Structure):
    _fields_ = _fields([("p", "k v page_table"), ("l", "layer_stride page_stride slot_stride head_stride"),
                        ("i", "layers num_pages page_size max_pages Hkv D dtype")])


class _Chunk(ctypes.Structure):
    _fields_ = _fields([("i", "B lead n_max"), ("p", "ctx_len n_nodes mask depths")])


class _AppendParams(ctypes.Structure):
    _fields_ = _fields([("p", "q k v q_out"), ("l", "q_stride k_stride v_stride q_out_stride"), ("i", "Hq"),
                        ("p", "q_norm k_norm"), ("f", "eps"), ("p", "freqs"), ("i", "rot_dim interleaved"),
                        ("f", "rot_scale"), ("i", "layer"), ("p", "stream")])


class _AttentionParams(ctypes.Structure):
    _fields_ = _fields([("p", "q out"), ("l", "q_stride out_stride"), ("i", "Hq"), ("f", "scale"), ("p", "lse"),
                        ("i", "layer"), ("p", "workspace"), ("z", "workspace_bytes"), ("p", "stream")])


class _LogitsParams(ctypes.Structure):
    _fields_ = _fields([("p", "logits out"), ("i", "B lead n_max V dtype"), ("p", "n_nodes history"),
                        ("i", "history_max"), ("p", "history_len prompt_len node_tokens node_mask repetition "
                                                    "frequency presence bias_ids bias"),
                        ("i", "n_bias"), ("p", "allow allow_index"), ("i", "allow_rows"), ("p", "stream")])


class _CommitParams(ctypes.Structure):
    _fields_ = _fields([("p", "tokens parents target"), ("i", "L"), ("p", "accepted lengths nodes stream")])


_pack_append, _pack_attention, _pack_logits, _pack_commit = (
    _packer(c) for c in (_AppendParams, _AttentionParams, _LogitsParams, _CommitParams))


class _TreeOut(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("parents", ctypes.c_void_p), ("depths", ctypes.c_void_p),
                ("scores", ctypes.c_void_p), ("mask", ctypes.c_void_p)]


EXPORTED = ("dt_build_tree", "dt_build_tree_noalloc", "dt_workspace_size", "dt_status_string", "dt_position_topk",
            "dt_ngram_update", "dt_verify_length", "dt_rope_frequencies", "dt_kv_append", "dt_tree_attention",
            "dt_attention_workspace", "dt_process_logits", "dt_commit_path")
DT_NOALLOC_SCRATCH_BYTES = 32 << 20

_lib = None


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() "
                              "(python -m draft_tree_construction_dt_amd.build)")
        lib = ctypes.CDLL(_LIB_PATH)
        lib.dt_build_tree.restype = ctypes.c_int
        lib.dt_build_tree.argtypes = [ctypes.c_void_p, ctypes.POINTER(_NGram), ctypes.POINTER(_Params),
                                      ctypes.POINTER(_TreeOut)]
        lib.dt_build_tree_noalloc.restype = ctypes.c_int
        lib.dt_build_tree_noalloc.argtypes = lib.dt_build_tree.argtypes
        lib.dt_workspace_size.restype = ctypes.c_size_t
        lib.dt_workspace_size.argtypes = [ctypes.POINTER(_Params)]
        lib.dt_status_string.restype = ctypes.c_char_p
        lib.dt_status_string.argtypes = [ctypes.c_int]
        lib.dt_position_topk.restype = ctypes.c_int
        lib.dt_position_topk.argtypes = [ctypes.c_void_p, ctypes.POINTER(_Params), ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p]
        lib.dt_ngram_update.restype = ctypes.c_int
        lib.dt_ngram_update.argtypes = [ctypes.POINTER(_NGram), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_int32, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p,
                                        ctypes.c_void_p]
        lib.dt_verify_length.restype = ctypes.c_int
        lib.dt_verify_length.argtypes = [ctypes.POINTER(_TreeOut), ctypes.c_int32, ctypes.c_int32, ctypes.c_double,
                                         ctypes.c_double, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        lib.dt_rope_frequencies.restype = ctypes.c_int
        lib.dt_rope_frequencies.argtypes = [ctypes.c_int32, ctypes.c_int32] + [ctypes.c_double] * 5 + \
            [ctypes.c_void_p, ctypes.POINTER(ctypes.c_float)]
        for fn in (lib.dt_kv_append, lib.dt_tree_attention, lib.dt_commit_path):
            fn.restype = ctypes.c_int
            fn.argtypes = [ctypes.c_void_p] * 3            # kv, chunk, params (a structure or its bytes)
        lib.dt_attention_workspace.restype = ctypes.c_size_t
        lib.dt_attention_workspace.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]
        lib.dt_process_logits.restype = ctypes.c_int
        lib.dt_process_logits.argtypes = [ctypes.c_void_p]
        _lib = lib
    return _lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# ---------------------------------------------------------------------------
# Python mirrors of the C structs (fields hold torch tensors or plain values)
# ---------------------------------------------------------------------------

@dataclass
class NGram:
    kind: int = DT_NGRAM_NONE
    min_logp: float = float("-inf")
    dense_logp: Optional[torch.Tensor] = None
    row_ptr: Optional[torch.Tensor] = None
    col: Optional[torch.Tensor] = None
    csr_logp: Optional[torch.Tensor] = None
    keys: Optional[torch.Tensor] = None      # int64 view of the uint64 keys
    succ: Optional[torch.Tensor] = None
    hash_logp: Optional[torch.Tensor] = None
    cap: int = 0
    S: int = 0

    def _c(self) -> _NGram:
        nnz = int(self.col.numel()) if isinstance(self.col, torch.Tensor) else 0
        return _NGram(int(self.kind), float(self.min_logp), _ptr(self.dense_logp), _ptr(self.row_ptr),
                      _ptr(self.col), _ptr(self.csr_logp), nnz, _ptr(self.keys), _ptr(self.succ),
                      _ptr(self.hash_logp), int(self.cap), int(self.S))


@dataclass
class Params:
    B: int
    V: int
    d: int
    k: int
    W: int
    budget: int
    dtype: int
    mode: int = DT_MODE_DART
    ctx: Optional[torch.Tensor] = None
    E: Optional[torch.Tensor] = None
    F: Optional[torch.Tensor] = None
    R: int = 0
    sweep_chunks: int = 0
    workspace: Optional[torch.Tensor] = None
    stream: Optional[object] = None           # torch.cuda.Stream, raw handle (int) or None = current
    prof_event_start: Optional[object] = None  # torch.cuda.Event or raw handle
    prof_event_stop: Optional[object] = None

    def _c(self) -> _Params:
        if self.stream is None:
            stream = torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else 0
        elif isinstance(self.stream, int):
            stream = self.stream
        else:
            stream = self.stream.cuda_stream

        def ev(e):
            if e is None:
                return None
            return e if isinstance(e, int) else e.cuda_event

        ws = self.workspace
        return _Params(int(self.B), int(self.V), int(self.d), int(self.k), int(self.W), int(self.budget),
                       int(self.dtype), int(self.mode), _ptr(self.ctx), _ptr(self.E), _ptr(self.F),
                       int(self.R), int(self.sweep_chunks), _ptr(ws),
                       int(ws.numel() * ws.element_size()) if ws is not None else 0,
                       stream, ev(self.prof_event_start), ev(self.prof_event_stop))


@dataclass
class TreeOut:
    n_nodes: torch.Tensor
    tokens: torch.Tensor
    parents: torch.Tensor
    depths: torch.Tensor
    scores: torch.Tensor
    mask: torch.Tensor

    def _c(self) -> _TreeOut:
        return _TreeOut(_ptr(self.n_nodes), _ptr(self.tokens), _ptr(self.parents), _ptr(self.depths),
                        _ptr(self.scores), _ptr(self.mask))

    def numpy(self) -> dict:
        return dict(n_nodes=self.n_nodes.cpu().numpy(), tokens=self.tokens.cpu().numpy(),
                    parents=self.parents.cpu().numpy(), depths=self.depths.cpu().numpy(),
                    scores=self.scores.cpu().numpy(),
                    mask=self.mask.cpu().numpy().view(np.uint32))


# ---------------------------------------------------------------------------
# the C entry points, same names
# ---------------------------------------------------------------------------

def dt_status_string(status: int) -> str:
    return _load().dt_status_string(int(status)).decode()


def dt_workspace_size(params: Params) -> int:
    p = params._c()
    return int(_load().dt_workspace_size(ctypes.byref(p)))


def dt_build_tree(logits: torch.Tensor, ngram: NGram, params: Params, out: TreeOut) -> None:
    g, p, o = ngram._c(), params._c(), out._c()
    st = _load().dt_build_tree(_ptr(logits), ctypes.byref(g), ctypes.byref(p), ctypes.byref(o))
    if st != DT_OK:
        raise DtError(st, "dt_build_tree")


def dt_build_tree_noalloc(logits: torch.Tensor, ngram: NGram, params: Params, out: TreeOut) -> None:
    """dt_build_tree on the library's own per-GPU scratch array (params.workspace
    is ignored): for callers that cannot allocate."""
    g, p, o = ngram._c(), params._c(), out._c()
    st = _load().dt_build_tree_noalloc(_ptr(logits), ctypes.byref(g), ctypes.byref(p), ctypes.byref(o))
    if st != DT_OK:
        raise DtError(st, "dt_build_tree_noalloc")


def dt_ngram_update(ngram: "NGram", ctx: torch.Tensor, tokens: torch.Tensor, lengths: torch.Tensor,
                    new_logp: float = 0.0, counts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Add the trigrams of the accepted tokens to a device trigram table in
    place (see dt_ngram_update in dt.h).  ctx int32 [B][2], tokens int32
    [B][L], lengths int32 [B], counts int32 [3] or None; all on the device."""
    g = ngram._c()
    B, L = (int(tokens.shape[0]), int(tokens.shape[1])) if tokens.dim() == 2 else (0, 0)
    if stream is None:
        h = torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else 0
    elif isinstance(stream, int):
        h = stream
    else:
        h = stream.cuda_stream
    st = _load().dt_ngram_update(ctypes.byref(g), _ptr(ctx), _ptr(tokens), _ptr(lengths), B, L,
                                 float(new_logp), _ptr(counts), h)
    if st != DT_OK:
        raise DtError(st, "dt_ngram_update")


def dt_verify_length(tree: "TreeOut", budget: int, cost_fixed: float, cost_per_token: float,
                     n_verify: torch.Tensor, rank: torch.Tensor, stream=None) -> None:
    """How many best-first nodes of each tree to verify, and every node's
    best-first position (see dt_verify_length in dt.h); all on the device."""
    t = tree._c()
    B = int(tree.n_nodes.shape[0])
    if stream is None:
        h = torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else 0
    elif isinstance(stream, int):
        h = stream
    else:
        h = stream.cuda_stream
    st = _load().dt_verify_length(ctypes.byref(t), B, int(budget), float(cost_fixed), float(cost_per_token),
                                  _ptr(n_verify), _ptr(rank), h)
    if st != DT_OK:
        raise DtError(st, "dt_verify_length")


def dt_position_topk(logits: torch.Tensor, params: Params, lse: torch.Tensor, topk_tok: torch.Tensor,
                     topk_val: torch.Tensor) -> None:
    p = params._c()
    st = _load().dt_position_topk(_ptr(logits), ctypes.byref(p), _ptr(lse), _ptr(topk_tok), _ptr(topk_val))
    if st != DT_OK:
        raise DtError(st, "dt_position_topk")


# ---------------------------------------------------------------------------
# the verification pass over a tree (second part of dt.h)
# ---------------------------------------------------------------------------

_HEAD_TYPES = {torch.bfloat16: DT_DTYPE_BF16, torch.float16: DT_DTYPE_F16}
_LOGIT_TYPES = {torch.float32: DT_DTYPE_F32, torch.bfloat16: DT_DTYPE_BF16}


def _need(ok: bool, where: str, what: str) -> None:
    """The C ABI sees addresses only: shapes, types and layouts are checked here."""
    if not ok:
        raise DtError(DT_ERR_INVALID_ARG, f"{where}: {what}")


def _at(t: Optional[torch.Tensor], shape, dtype, index: int, where: str, name: str) -> int:
    """Address of a contiguous tensor of this shape, type and device (get_device()); 0 without one."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise DtError(DT_ERR_INVALID_ARG,
                      f"{where}: {name} must be contiguous {dtype} {tuple(shape)} on the call's device, "
                      f"not {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, index: int) -> int:
    """Raw handle of `stream`, which must be the device's, or of its current one."""
    if isinstance(stream, int):
        return stream
    if stream is not None:
        _need(index < 0 or stream.device_index == index, "stream", "must belong to the tensors' device")
        return stream.cuda_stream
    if index < 0:
        return 0
    return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_device(index: int, call, *args):
    """call(*args) with device `index` current: the handle of a device's
    default stream is null, which the C ABI takes for the current device's."""
    if index < 0 or _current_device() == index:
        return call(*args)
    with torch.cuda.device(index):
        return call(*args)


def _reachable(index: int, B: int, call):
    """`call`, or a refusal in its place where the tensors lie in host memory,
    which kernels cannot reach (an empty batch launches none)."""
    if index >= 0 or B == 0:
        return call

    def refuse(*_):
        raise DtError(DT_ERR_INVALID_ARG, f"{refuse.__name__}: the tensors must be on a GPU")

    refuse.__name__ = call.__name__
    return refuse


class KVCache:
    """A paged cache of keys and values (dt_kv_cache): k and v of shape
    [pages][page_size][Hkv][D], or [layers][pages][page_size][Hkv][D] for one
    allocation of all layers, bf16 or f16, with equal strides and contiguous
    heads (a [pages][Hkv][page_size][D] pool is passed as its
    ``transpose(-3, -2)``); page_table int32 [B][max_pages].  Holds the
    tensors; make another for other tensors."""

    __slots__ = ("k", "v", "page_table", "device", "index", "dtype", "Hkv", "D", "layers", "_struct", "_ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor):
        w = "KVCache"
        _need(k.dim() in (4, 5), w, "k must be [pages][page_size][Hkv][D] or [layers][pages][page_size][Hkv][D]")
        _need(v.shape == k.shape and v.stride() == k.stride(), w, "v must have k's shape and strides")
        _need(k.dtype in _HEAD_TYPES and v.dtype == k.dtype, w, "k and v must be bfloat16 or float16")
        _need(k.stride(-1) == 1, w, "heads must be contiguous")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.is_contiguous(), w,
              "page_table must be contiguous int32 [B][max_pages]")
        _need(v.device == k.device and page_table.device == k.device, w, "k, v and page_table on one device")
        self.k, self.v, self.page_table = k, v, page_table
        self.device, self.dtype, self.Hkv, self.D = k.device, k.dtype, int(k.shape[-2]), int(k.shape[-1])
        self.layers, self.index = int(k.shape[0]) if k.dim() == 5 else 1, k.get_device()
        self._struct = _KVCache(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), k.stride(0) if k.dim() == 5 else 0,
                                k.stride(-4), k.stride(-3), k.stride(-2), self.layers, k.shape[-4], k.shape[-3],
                                page_table.shape[1], self.Hkv, self.D, _HEAD_TYPES[k.dtype])
        self._ref = ctypes.addressof(self._struct)


class Chunk:
    """The new tokens of a batch (dt_chunk): per request `lead` committed
    tokens and up to n_max tree nodes.  ctx_len and n_nodes int32 [B]; mask
    and depths as dt_build_tree wrote them for a budget of n_max
    (``Chunk.of_tree``).  Holds the tensors, whose values may change between
    calls; make another for other tensors."""

    __slots__ = ("ctx_len", "n_nodes", "mask", "depths", "B", "lead", "n_max", "rows", "device", "index", "_struct",
                 "_ref")

    def __init__(self, ctx_len: torch.Tensor, lead: int = 1, n_max: int = 0, n_nodes: Optional[torch.Tensor] = None,
                 mask: Optional[torch.Tensor] = None, depths: Optional[torch.Tensor] = None):
        w, dev = "Chunk", ctx_len.get_device()
        _need(ctx_len.dim() == 1, w, "ctx_len must be int32 [B]")
        B, n_max, lead = int(ctx_len.shape[0]), int(n_max), int(lead)
        _at(ctx_len, (B,), torch.int32, dev, w, "ctx_len")
        _at(n_nodes, (B,), torch.int32, dev, w, "n_nodes")
        _at(mask, (B, n_max, (n_max + 31) // 32), torch.int32, dev, w, "mask")
        _at(depths, (B, n_max), torch.int32, dev, w, "depths")
        self.ctx_len, self.n_nodes, self.mask, self.depths = ctx_len, n_nodes, mask, depths
        self.B, self.lead, self.n_max, self.rows = B, lead, n_max, lead + n_max
        self.device, self.index = ctx_len.device, dev
        self._struct = _Chunk(B, lead, n_max, _ptr(ctx_len), _ptr(n_nodes), _ptr(mask), _ptr(depths))
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def of_tree(cls, ctx_len: torch.Tensor, tree: TreeOut, lead: int = 1) -> "Chunk":
        """The chunk of built trees behind `lead` committed tokens."""
        return cls(ctx_len, lead, int(tree.tokens.shape[1]), tree.n_nodes, tree.mask, tree.depths)


def _row_stride(t: Optional[torch.Tensor], shape, kv: KVCache, where: str, name: str) -> int:
    """Row stride of a [B][rows][H][D] tensor whose rows' heads are contiguous."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not kv.dtype or t.get_device() != kv.index:
        raise DtError(DT_ERR_INVALID_ARG, f"{where}: {name} must be {kv.dtype} [B][lead + n_max][heads][D] = "
                                          f"{tuple(shape)} on the cache's device, not {t.dtype} {tuple(t.shape)}")
    batch, row, head, one = t.stride()
    if one != 1 or (head != kv.D and shape[2] != 1):
        raise DtError(DT_ERR_INVALID_ARG, f"{where}: the heads of a row of {name} must be contiguous")
    if shape[0] == 1:
        return row
    if shape[1] == 1:
        return batch
    if batch != shape[1] * row:
        raise DtError(DT_ERR_INVALID_ARG, f"{where}: the rows of {name} must be evenly spaced over the batch")
    return row


def _pass_devices(kv: Optional[KVCache], chunk: Chunk, where: str) -> None:
    _need(kv is None or (chunk.index == kv.index and kv.page_table.shape[0] >= chunk.B), where,
          "the chunk and the cache must be on one device, with a row of page_table for every request")


def dt_rope_frequencies(rot_dim: int, base: float, kind: int = DT_ROPE_NONE, factor: float = 1.0, low: float = 1.0,
                        high: float = 32.0, original: float = 4096.0):
    """(float64 CPU tensor [rot_dim / 2] of radians a position, rot_scale) of
    rotary positions, scaled for long contexts by `kind`."""
    freqs = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float64)
    scale = ctypes.c_float()
    st = _load().dt_rope_frequencies(int(kind), int(rot_dim), float(base), float(factor), float(low), float(high),
                                     float(original), freqs.data_ptr(), ctypes.byref(scale))
    if st != DT_OK:
        raise DtError(st, "dt_rope_frequencies")
    return freqs, scale.value


def dt_kv_append(kv: KVCache, chunk: Chunk, k: torch.Tensor, v: torch.Tensor, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6, freqs: Optional[torch.Tensor] = None,
                 interleaved: bool = False, rot_scale: float = 1.0, layer: int = 0, stream=None) -> None:
    """Norm and turn the chunk's queries and keys, put keys and values into
    the cache (see dt_kv_append in dt.h).  q, k, v, q_out [B][lead + n_max]
    [heads][D], evenly spaced rows (slices of one projection); q_norm and
    k_norm [D]; freqs float64 [rot_dim / 2] on the device."""
    w, index, dtype = "dt_kv_append", kv.index, kv.dtype
    _pass_devices(kv, chunk, w)
    B, rows, D, Hq = chunk.B, chunk.rows, kv.D, 0
    if q is not None:
        _need(q.dim() == 4, w, "q must be [B][lead + n_max][heads][D]")
        Hq = int(q.shape[2])
    heads, kv_heads = (B, rows, Hq, D), (B, rows, kv.Hkv, D)
    call = _reachable(index, B, _load().dt_kv_append)
    st = _on_device(index, call, kv._ref, chunk._ref, _pack_append(
        0 if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), 0 if q_out is None else q_out.data_ptr(),
        _row_stride(q, heads, kv, w, "q"), _row_stride(k, kv_heads, kv, w, "k"), _row_stride(v, kv_heads, kv, w, "v"),
        _row_stride(q_out, heads, kv, w, "q_out"), Hq, _at(q_norm, (D,), dtype, index, w, "q_norm"),
        _at(k_norm, (D,), dtype, index, w, "k_norm"), eps,
        0 if freqs is None else _at(freqs, (freqs.numel(),), torch.float64, index, w, "freqs"),
        0 if freqs is None else 2 * freqs.numel(), bool(interleaved), rot_scale, layer, _stream_of(stream, index)))
    if st != DT_OK:
        raise DtError(st, w)


def dt_attention_workspace(kv: KVCache, chunk: Chunk, Hq: int) -> int:
    return int(_load().dt_attention_workspace(kv._ref, chunk._ref, int(Hq)))


def dt_tree_attention(kv: KVCache, chunk: Chunk, q: torch.Tensor, out: torch.Tensor, scale: Optional[float] = None,
                      lse: Optional[torch.Tensor] = None, layer: int = 0, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """Attention of the chunk's rows over the cache (see dt_tree_attention in
    dt.h).  q and out [B][lead + n_max][Hq][D]; scale defaults to D^-1/2; lse
    float32 [B][lead + n_max][Hq] or None; workspace of
    dt_attention_workspace() bytes."""
    w, index = "dt_tree_attention", kv.index
    _pass_devices(kv, chunk, w)
    _need(q.dim() == 4, w, "q must be [B][lead + n_max][heads][D]")
    Hq = int(q.shape[2])
    heads = (chunk.B, chunk.rows, Hq, kv.D)
    _need(workspace is None or (workspace.get_device() == index and workspace.is_contiguous()), w,
          "workspace must be contiguous, on the cache's device")
    call = _reachable(index, chunk.B, _load().dt_tree_attention)
    st = _on_device(index, call, kv._ref, chunk._ref, _pack_attention(
        q.data_ptr(), out.data_ptr(), _row_stride(q, heads, kv, w, "q"), _row_stride(out, heads, kv, w, "out"), Hq,
        kv.D ** -0.5 if scale is None else scale, _at(lse, heads[:3], torch.float32, index, w, "lse"), layer,
        0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
        _stream_of(stream, index)))
    if st != DT_OK:
        raise DtError(st, w)


def dt_process_logits(logits: torch.Tensor, out: torch.Tensor, history: Optional[torch.Tensor] = None,
                      history_len: Optional[torch.Tensor] = None, prompt_len: Optional[torch.Tensor] = None,
                      repetition: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                      presence: Optional[torch.Tensor] = None, bias_ids: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, allow: Optional[torch.Tensor] = None,
                      allow_index: Optional[torch.Tensor] = None, lead: Optional[int] = None,
                      n_nodes: Optional[torch.Tensor] = None, node_tokens: Optional[torch.Tensor] = None,
                      node_mask: Optional[torch.Tensor] = None, stream=None) -> None:
    """Penalties, biases and grammar masks on logits [B][lead + n_max][V]
    (see dt_process_logits in dt.h).  lead defaults to every row (draft
    positions, no tree).  history int32 [B][history_max]; bias_ids int32 and
    bias float32 [B][n_bias]; allow int32 [allow_rows][ceil(V/32)];
    allow_index int32 [B][lead + n_max]; the rest [B]."""
    w, dev = "dt_process_logits", logits.get_device()
    _need(logits.dim() == 3 and logits.dtype in _LOGIT_TYPES, w, "logits must be float32 or bfloat16 [B][rows][V]")
    B, rows, V = logits.shape
    lead = rows if lead is None else int(lead)
    n_max, i32, f32, each = rows - lead, torch.int32, torch.float32, (B,)
    _need(0 <= lead <= rows, w, "lead must be 0..rows")
    for t, name in ((history, "history"), (bias_ids, "bias_ids"), (allow, "allow")):
        _need(t is None or t.dim() == 2, w, f"{name} must have two axes")
    hmax = 0 if history is None else history.shape[1]
    nb = 0 if bias_ids is None else bias_ids.shape[1]
    arows = 0 if allow is None else allow.shape[0]
    call = _reachable(dev, B, _load().dt_process_logits)
    st = _on_device(dev, call, _pack_logits(
        _at(logits, logits.shape, logits.dtype, dev, w, "logits"), _at(out, logits.shape, logits.dtype, dev, w, "out"),
        B, lead, n_max, V, _LOGIT_TYPES[logits.dtype],
        _at(n_nodes, each, i32, dev, w, "n_nodes"), _at(history, (B, hmax), i32, dev, w, "history"), hmax,
        _at(history_len, each, i32, dev, w, "history_len"), _at(prompt_len, each, i32, dev, w, "prompt_len"),
        _at(node_tokens, (B, n_max), i32, dev, w, "node_tokens"),
        _at(node_mask, (B, n_max, (n_max + 31) // 32), i32, dev, w, "node_mask"),
        _at(repetition, each, f32, dev, w, "repetition"), _at(frequency, each, f32, dev, w, "frequency"),
        _at(presence, each, f32, dev, w, "presence"), _at(bias_ids, (B, nb), i32, dev, w, "bias_ids"),
        _at(bias, (B, nb), f32, dev, w, "bias"), nb, _at(allow, (arows, (V + 31) // 32), i32, dev, w, "allow"),
        _at(allow_index, (B, rows), i32, dev, w, "allow_index"), arows, _stream_of(stream, dev)))
    if st != DT_OK:
        raise DtError(st, w)


def dt_commit_path(kv: Optional[KVCache], chunk: Chunk, tokens: Optional[torch.Tensor],
                   parents: Optional[torch.Tensor], target: torch.Tensor, accepted: torch.Tensor,
                   lengths: torch.Tensor, nodes: Optional[torch.Tensor] = None, stream=None) -> None:
    """Accept each tree's path along the target's choices and move its keys
    and values, in every layer, to the front of the chunk's slots (see
    dt_commit_path in dt.h).  tokens and parents int32 [B][n_max] as
    dt_build_tree wrote them; target int32 [B][lead + n_max]; accepted and
    nodes int32 [B][L], lengths int32 [B] are written."""
    w, dev, i32 = "dt_commit_path", chunk.index, torch.int32
    _pass_devices(kv, chunk, w)
    _need(accepted.dim() == 2, w, "accepted must be int32 [B][L]")
    B, L = chunk.B, accepted.shape[1]
    call = _reachable(dev, B, _load().dt_commit_path)
    st = _on_device(dev, call, 0 if kv is None else kv._ref, chunk._ref, _pack_commit(
        _at(tokens, (B, chunk.n_max), i32, dev, w, "tokens"), _at(parents, (B, chunk.n_max), i32, dev, w, "parents"),
        _at(target, (B, chunk.rows), i32, dev, w, "target"), L, _at(accepted, (B, L), i32, dev, w, "accepted"),
        _at(lengths, (B,), i32, dev, w, "lengths"), _at(nodes, (B, L), i32, dev, w, "nodes"), _stream_of(stream, dev)))
    if st != DT_OK:
        raise DtError(st, w)


# ---------------------------------------------------------------------------
# plumbing: move a generated problem to the device and allocate outputs
# ---------------------------------------------------------------------------

def _dev(a, device, dtype=None):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint64:
        a = a.view(np.int64)
    elif a.dtype == np.uint16:
        a = a.view(np.int16)
    t = torch.from_numpy(a)
    if dtype is not None:
        t = t.to(dtype)
    return t.to(device)


def upload_ngram(ng, device) -> NGram:
    return NGram(kind=int(ng.kind), min_logp=float(ng.min_logp),
                 dense_logp=_dev(ng.dense_logp, device), row_ptr=_dev(ng.row_ptr, device),
                 col=_dev(ng.col, device), csr_logp=_dev(ng.csr_logp, device),
                 keys=_dev(ng.keys, device), succ=_dev(ng.succ, device),
                 hash_logp=_dev(ng.hash_logp, device), cap=int(ng.cap or 0), S=int(ng.S or 0))


def alloc_tree_out(B: int, budget: int, device) -> TreeOut:
    words = (budget + 31) // 32
    i32 = dict(dtype=torch.int32, device=device)
    return TreeOut(n_nodes=torch.empty(B, **i32), tokens=torch.empty(B, budget, **i32),
                   parents=torch.empty(B, budget, **i32), depths=torch.empty(B, budget, **i32),
                   scores=torch.empty(B, budget, dtype=torch.float32, device=device),
                   mask=torch.empty(B, budget, words, **i32))


def logits_tensor(p, device) -> torch.Tensor:
    if p.logits.dtype == np.uint16:
        return _dev(p.logits, device).view(torch.bfloat16)
    return _dev(p.logits, device, torch.float32)


@dataclass
class DeviceProblem:
    logits: torch.Tensor
    ngram: NGram
    params: Params
    out: TreeOut
    extra_logits: list = field(default_factory=list)


def upload_problem(p, device, *, sweep_chunks: int = 0, W=None, budget=None) -> DeviceProblem:
    """Copy a generated problem to ``device`` and size the workspace and outputs."""
    W = p.W if W is None else W
    budget = p.budget if budget is None else budget
    dtype = DT_DTYPE_BF16 if p.logits.dtype == np.uint16 else DT_DTYPE_F32
    params = Params(B=p.B, V=p.V, d=p.d, k=p.k, W=W, budget=budget, dtype=dtype, mode=int(p.mode),
                    ctx=_dev(p.ctx, device, torch.int32), E=_dev(p.E, device), F=_dev(p.F, device),
                    R=int(p.R or 0), sweep_chunks=sweep_chunks)
    nbytes = dt_workspace_size(params)
    params.workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    return DeviceProblem(logits=logits_tensor(p, device), ngram=upload_ngram(p.ngram, device),
                         params=params, out=alloc_tree_out(p.B, budget, device))
