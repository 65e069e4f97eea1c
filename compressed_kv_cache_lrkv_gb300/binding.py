"""Thin ctypes binding of liblrkv.so (include/lrkv.h): argument marshalling only.

Every function here forwards to the C entry point of the same name; tensors
are torch CUDA tensors whose data pointers are passed through.  Nothing is
computed in Python, and there is no fallback: if the library cannot be loaded
(or a call returns an error) an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

LRKV_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "workspace too small", 4: "CUDA error",
                5: "device bounds", 6: "timeout"}
DEV_BAD_BLOCK, DEV_BAD_SEQLEN, DEV_BAD_SLOT, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEV_NO_PAGES, DEV_BAD_INDEX = 0x10, 0x20

EXPORTED = ["lrkv_abi_version", "lrkv_status_string", "lrkv_last_error", "lrkv_cache_block_bytes", "lrkv_append",
            "lrkv_decode_workspace_bytes", "lrkv_decode", "lrkv_decode_fused", "lrkv_decode_static_ws",
            "lrkv_decode_partials", "lrkv_decode_merge",
            "lrkv_append_layers", "lrkv_decode_layers",
            "lrkv_prefill_workspace_bytes", "lrkv_prefill", "lrkv_prefill_fused", "lrkv_mla_cache_block_bytes", "lrkv_mla_append",
            "lrkv_mla_decode_workspace_bytes", "lrkv_mla_decode", "lrkv_train_forward", "lrkv_train_workspace_bytes",
            "lrkv_train_backward", "lrkv_quant_row_bytes", "lrkv_quant_block_bytes", "lrkv_cache_quantize",
            "lrkv_cache_dequantize", "lrkv_decode_quant_workspace_bytes", "lrkv_decode_quant",
            "lrkv_decode_quant_partials", "lrkv_decode_shared_workspace_bytes", "lrkv_decode_shared",
            "lrkv_prefix_partials", "lrkv_decode_tree_workspace_bytes", "lrkv_decode_tree", "lrkv_rope_make_plan",
            "lrkv_rope", "lrkv_pages_reserve", "lrkv_pages_fork", "lrkv_pages_free", "lrkv_pages_copy",
            "lrkv_cache_compact"]
MAX_TREE = 64  # LRKV_MAX_TREE
STATIC_WS_BYTES = 16 << 20  # LRKV_STATIC_WS_BYTES


class LrkvError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d_h", ctypes.c_int32), ("r", ctypes.c_int32), ("d", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("d_rope", ctypes.c_int32),
                ("rope_base", ctypes.c_float), ("num_splits", ctypes.c_int32)]


class LayerStrides(ctypes.Structure):
    """Element strides between consecutive layers' tensors (lrkv_layer_strides)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("X", "W_catT", "q", "BK", "BV", "out", "sK", "sV", "zK", "zV")]


class MlaDims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d_c", ctypes.c_int32), ("d_rope", ctypes.c_int32), ("d_head", ctypes.c_int32),
                ("d", ctypes.c_int32), ("block_size", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("rope_base", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("sK", ctypes.c_void_p), ("sV", ctypes.c_void_p), ("zK", ctypes.c_void_p), ("zV", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32)]


class QuantCacheStruct(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("num_blocks", ctypes.c_int32)]


class RopeSpec(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("d_rot", "layout", "scaling", "reserved")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "original_len", "low", "high", "magnitude")]


class RopePlan(ctypes.Structure):
    """Speeds of a rotation (lrkv_rope_plan), made by rope_plan."""
    _fields_ = [("d_rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turn", ctypes.c_uint64 * 128)]


class RowsStruct(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("num_rows", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("index", ctypes.c_void_p)]


class PoolsStruct(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p * 4), ("row_bytes", ctypes.c_int64 * 4), ("layer_bytes", ctypes.c_int64 * 4),
                ("num_pools", ctypes.c_int32), ("num_layers", ctypes.c_int32), ("num_blocks", ctypes.c_int32)]


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load (building first if needed) liblrkv.so and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        path = _build.build()
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    P = ctypes.POINTER
    lib.lrkv_abi_version.restype = ctypes.c_int
    lib.lrkv_status_string.restype = ctypes.c_char_p
    lib.lrkv_status_string.argtypes = [ctypes.c_int]
    lib.lrkv_last_error.restype = ctypes.c_char_p
    lib.lrkv_cache_block_bytes.restype = sz
    lib.lrkv_cache_block_bytes.argtypes = [P(Dims)]
    lib.lrkv_append.restype = ctypes.c_int
    lib.lrkv_append.argtypes = [P(Dims), vp, vp, i32, vp, vp, P(Cache), vp, vp]
    lib.lrkv_decode_workspace_bytes.restype = sz
    lib.lrkv_decode_workspace_bytes.argtypes = [P(Dims), i32]
    lib.lrkv_decode.restype = ctypes.c_int
    lib.lrkv_decode.argtypes = [P(Dims), vp, vp, vp, P(Cache), vp, i32, vp, i32, vp, vp, sz, vp, vp]
    lib.lrkv_decode_fused.restype = ctypes.c_int
    lib.lrkv_decode_fused.argtypes = [P(Dims), vp, vp, P(Cache), vp, i32, vp, i32, vp, vp, sz, vp, vp]
    lib.lrkv_append_layers.restype = ctypes.c_int
    lib.lrkv_append_layers.argtypes = [P(Dims), i32, P(LayerStrides), vp, vp, i32, vp, vp, P(Cache), vp, vp]
    lib.lrkv_decode_layers.restype = ctypes.c_int
    lib.lrkv_decode_layers.argtypes = [P(Dims), i32, P(LayerStrides), vp, vp, vp, P(Cache), vp, i32, vp, i32, vp, vp,
                                       sz, vp, vp]
    lib.lrkv_decode_partials.restype = ctypes.c_int
    lib.lrkv_decode_partials.argtypes = [P(Dims), vp, vp, P(Cache), vp, i32, vp, i32, vp, vp, sz, vp, vp]
    lib.lrkv_decode_merge.restype = ctypes.c_int
    lib.lrkv_decode_merge.argtypes = [P(Dims), i32, vp, vp, i32, vp, vp, vp]
    lib.lrkv_decode_static_ws.restype = ctypes.c_int
    lib.lrkv_decode_static_ws.argtypes = [P(Dims), vp, vp, vp, P(Cache), vp, i32, vp, i32, vp, vp, vp]
    lib.lrkv_prefill_workspace_bytes.restype = sz
    lib.lrkv_prefill_workspace_bytes.argtypes = [P(Dims), i32, i32]
    lib.lrkv_prefill.restype = ctypes.c_int
    lib.lrkv_prefill.argtypes = [P(Dims), vp, vp, vp, P(Cache), vp, i32, vp, i32, i32, vp, vp, sz, vp, vp]
    lib.lrkv_prefill_fused.restype = ctypes.c_int
    lib.lrkv_prefill_fused.argtypes = [P(Dims), vp, vp, P(Cache), vp, i32, vp, i32, i32, vp, vp, vp]
    lib.lrkv_train_forward.restype = ctypes.c_int
    lib.lrkv_train_forward.argtypes = [P(Dims), vp, vp, vp, i32, vp, vp, vp, vp]
    lib.lrkv_train_workspace_bytes.restype = sz
    lib.lrkv_train_workspace_bytes.argtypes = [P(Dims), i32]
    lib.lrkv_train_backward.restype = ctypes.c_int
    lib.lrkv_train_backward.argtypes = [P(Dims), vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, sz, vp, vp]
    lib.lrkv_mla_cache_block_bytes.restype = sz
    lib.lrkv_mla_cache_block_bytes.argtypes = [P(MlaDims)]
    lib.lrkv_mla_append.restype = ctypes.c_int
    lib.lrkv_mla_append.argtypes = [P(MlaDims), vp, vp, i32, vp, vp, vp, i32, vp, vp]
    lib.lrkv_mla_decode_workspace_bytes.restype = sz
    lib.lrkv_mla_decode_workspace_bytes.argtypes = [P(MlaDims), i32]
    lib.lrkv_mla_decode.restype = ctypes.c_int
    lib.lrkv_mla_decode.argtypes = [P(MlaDims), vp, vp, i32, vp, i32, vp, i32, vp, vp, sz, vp, vp]
    for f in (lib.lrkv_quant_row_bytes, lib.lrkv_quant_block_bytes):
        f.restype, f.argtypes = sz, [P(Dims)]
    lib.lrkv_cache_quantize.restype = ctypes.c_int
    lib.lrkv_cache_quantize.argtypes = [P(Dims), i32, P(Cache), vp, P(QuantCacheStruct), vp, vp, vp]
    lib.lrkv_cache_dequantize.restype = ctypes.c_int
    lib.lrkv_cache_dequantize.argtypes = [P(Dims), i32, P(QuantCacheStruct), vp, P(Cache), vp, vp, vp]
    lib.lrkv_decode_quant_workspace_bytes.restype = sz
    lib.lrkv_decode_quant_workspace_bytes.argtypes = [P(Dims), i32]
    lib.lrkv_decode_quant.restype = ctypes.c_int
    lib.lrkv_decode_quant.argtypes = [P(Dims), vp, vp, vp, P(QuantCacheStruct), vp, i32, vp, i32, vp, vp, sz, vp, vp]
    lib.lrkv_decode_quant_partials.restype = ctypes.c_int
    lib.lrkv_decode_quant_partials.argtypes = [P(Dims), vp, vp, P(QuantCacheStruct), vp, i32, vp, i32, vp, vp, sz, vp,
                                               vp]
    lib.lrkv_decode_shared_workspace_bytes.restype = sz
    lib.lrkv_decode_shared_workspace_bytes.argtypes = [P(Dims), i32, i32]
    lib.lrkv_decode_shared.restype = ctypes.c_int
    lib.lrkv_decode_shared.argtypes = [P(Dims), vp, vp, vp, P(Cache), vp, i32, vp, vp, i32, vp, i32, vp, vp, sz, vp,
                                       vp]
    lib.lrkv_prefix_partials.restype = ctypes.c_int
    lib.lrkv_prefix_partials.argtypes = [P(Dims), vp, vp, P(Cache), vp, i32, vp, i32, vp, vp, sz, vp, vp]
    lib.lrkv_decode_tree_workspace_bytes.restype = sz
    lib.lrkv_decode_tree_workspace_bytes.argtypes = [P(Dims), i32, i32]
    lib.lrkv_rope_make_plan.argtypes = [P(RopeSpec), P(RopePlan)]
    lib.lrkv_decode_tree.argtypes = [P(Dims), vp, vp, vp, P(Cache), vp, i32, vp, vp, vp, i32, i32, vp, vp, sz, vp, vp]
    lib.lrkv_rope.argtypes = [P(RopePlan), i32, i32, i32, i32, i32, P(RowsStruct), P(RowsStruct), vp, i32, vp, vp]
    lib.lrkv_pages_reserve.argtypes = [i32, vp, vp, i32, vp, vp, i32, vp, vp]
    lib.lrkv_pages_fork.argtypes = [P(PoolsStruct), vp, vp, i32, vp, i32, vp, vp, i32, vp, vp]
    lib.lrkv_pages_free.argtypes = [i32, vp, vp, i32, vp, i32, vp, i32, vp, vp, vp]
    lib.lrkv_pages_copy.argtypes = [P(PoolsStruct), vp, P(PoolsStruct), vp, i32, vp, vp]
    lib.lrkv_cache_compact.argtypes = [P(PoolsStruct), vp, i32, vp, i32, vp, vp, i32, vp, vp, vp]
    for f in (lib.lrkv_rope_make_plan, lib.lrkv_decode_tree, lib.lrkv_rope, lib.lrkv_pages_reserve,
              lib.lrkv_pages_fork, lib.lrkv_pages_free, lib.lrkv_pages_copy, lib.lrkv_cache_compact):
        f.restype = ctypes.c_int
    _lib = lib
    return lib


def make_dims(H: int, d_h: int, r: int, d: int, block_size: int = 64, softmax_scale: float = 0.0, d_rope: int = 0,
              rope_base: float = 0.0, num_splits: int = 0) -> Dims:
    return Dims(H, d_h, r, d, block_size, softmax_scale, d_rope, rope_base, num_splits)


def make_mla_dims(H: int, d: int, d_head: int = 128, d_c: int = 512, d_rope: int = 64, block_size: int = 64,
                  softmax_scale: float = 0.0, rope_base: float = 0.0) -> MlaDims:
    return MlaDims(H, d_c, d_rope, d_head, d, block_size, softmax_scale, rope_base)


def _ptr(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without a Stream object around it (0.3 us a call instead of 3), and the current device's
# number as torch.cuda.current_device() asks for it (0.2 us less).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != LRKV_OK:
        raise LrkvError(rc, where, load().lrkv_last_error().decode())


class PagedCache:
    """One layer's four cache pools (device tensors, bf16 bit patterns as int16/bfloat16)."""

    def __init__(self, sK, sV, zK, zV):
        self.sK, self.sV, self.zK, self.zV = sK, sV, zK, zV
        self.num_blocks = int(sK.shape[0])

    @classmethod
    def empty(cls, num_blocks: int, H: int, d_h: int, r: int, block_size: int = 64, device="cuda", d_rope: int = 0):
        mk = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=device)
        return cls(mk(num_blocks, block_size, d_h + d_rope), mk(num_blocks, block_size, d_h),
                   mk(num_blocks, block_size, H, r), mk(num_blocks, block_size, H, r))

    def struct(self) -> Cache:
        return Cache(_ptr(self.sK), _ptr(self.sV), _ptr(self.zK), _ptr(self.zV), self.num_blocks)

    def tensors(self):
        return self.sK, self.sV, self.zK, self.zV


def abi_version() -> int:
    return int(load().lrkv_abi_version())


def cache_block_bytes(dims: Dims) -> int:
    return int(load().lrkv_cache_block_bytes(ctypes.byref(dims)))


def decode_workspace_bytes(dims: Dims, batch: int) -> int:
    return int(load().lrkv_decode_workspace_bytes(ctypes.byref(dims), batch))


def prefill_workspace_bytes(dims: Dims, batch: int, Tq: int) -> int:
    return int(load().lrkv_prefill_workspace_bytes(ctypes.byref(dims), batch, Tq))


def lrkv_append(dims: Dims, X, W_catT, slot_mapping, cache: PagedCache, status=None, stream=None, positions=None):
    """Eqs. (4)-(5): write rows of X [n, d] into the cache at slot_mapping [n]; with a
    positional key (dims.d_rope > 0) its columns are rotated at positions [n] (int32)."""
    n = int(X.shape[0])
    c = cache.struct()
    rc = load().lrkv_append(ctypes.byref(dims), _ptr(X), _ptr(W_catT), n, _ptr(slot_mapping), _ptr(positions),
                            ctypes.byref(c), _ptr(status), _stream(stream))
    _check(rc, "lrkv_append")


def lrkv_decode(dims: Dims, q, BK, BV, cache: PagedCache, block_table, seq_lens, out, workspace, status=None,
                stream=None):
    """Factored decode (Eqs. (6)-(7)): q [B, H, d_h] -> out [B, H, d_h]."""
    B = int(q.shape[0])
    c = cache.struct()
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().lrkv_decode(ctypes.byref(dims), _ptr(q), _ptr(BK), _ptr(BV), ctypes.byref(c), _ptr(block_table),
                            int(block_table.shape[1]), _ptr(seq_lens), B, _ptr(out), _ptr(workspace), ws_bytes,
                            _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode")


def lrkv_decode_fused(dims: Dims, q, q_tilde, cache: PagedCache, block_table, seq_lens, out, workspace, status=None,
                      stream=None):
    """Decode with absorbed weights: q [B, H, d_h], q~ [B, H, r] -> out [B, H, d_h + r] = [o_s | o_z]."""
    B = int(q.shape[0])
    c = cache.struct()
    rc = load().lrkv_decode_fused(ctypes.byref(dims), _ptr(q), _ptr(q_tilde), ctypes.byref(c), _ptr(block_table),
                                  int(block_table.shape[1]), _ptr(seq_lens), B, _ptr(out), _ptr(workspace),
                                  int(workspace.numel() * workspace.element_size()), _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_fused")


def lrkv_decode_partials(dims: Dims, q, BK, cache: PagedCache, block_table, seq_lens, partials, workspace,
                         status=None, stream=None):
    """Decode partials over this cache's tokens: q [B, H, d_h] -> partials [B, H, d_h + r + 2] fp32
    (acc_s, acc_z, m, l)."""
    B = int(q.shape[0])
    c = cache.struct()
    rc = load().lrkv_decode_partials(ctypes.byref(dims), _ptr(q), _ptr(BK), ctypes.byref(c), _ptr(block_table),
                                     int(block_table.shape[1]), _ptr(seq_lens), B, _ptr(partials), _ptr(workspace),
                                     int(workspace.numel() * workspace.element_size()), _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_partials")


def lrkv_decode_merge(dims: Dims, partials, BV, out, status=None, stream=None):
    """Merge partials [P, B, H, d_h + r + 2] of P parts of the sequences' tokens -> out [B, H, d_h]."""
    P, B = int(partials.shape[0]), int(partials.shape[1])
    rc = load().lrkv_decode_merge(ctypes.byref(dims), P, _ptr(partials), _ptr(BV), B, _ptr(out), _ptr(status),
                                  _stream(stream))
    _check(rc, "lrkv_decode_merge")


def lrkv_decode_static_ws(dims: Dims, q, BK, BV, cache: PagedCache, block_table, seq_lens, out, status=None,
                          stream=None):
    """lrkv_decode with the library's static scratch area instead of a caller
    workspace, for callers that must not allocate device memory (see lrkv.h)."""
    B = int(q.shape[0])
    c = cache.struct()
    rc = load().lrkv_decode_static_ws(ctypes.byref(dims), _ptr(q), _ptr(BK), _ptr(BV), ctypes.byref(c),
                                      _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), B, _ptr(out),
                                      _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_static_ws")


class LayeredCache:
    """Several layers' cache pools as tensors with a leading layer dimension
    ([layers, num_blocks, block_size, ...]); layer l is at l * stride(0) elements."""

    def __init__(self, sK, sV, zK, zV):
        self.sK, self.sV, self.zK, self.zV = sK, sV, zK, zV
        self.num_layers = int(sK.shape[0])
        self.num_blocks = int(sK.shape[1])

    @classmethod
    def empty(cls, num_layers: int, num_blocks: int, H: int, d_h: int, r: int, block_size: int = 64, device="cuda",
              d_rope: int = 0):
        mk = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=device)
        return cls(mk(num_layers, num_blocks, block_size, d_h + d_rope), mk(num_layers, num_blocks, block_size, d_h),
                   mk(num_layers, num_blocks, block_size, H, r), mk(num_layers, num_blocks, block_size, H, r))

    def struct(self) -> Cache:
        return Cache(_ptr(self.sK), _ptr(self.sV), _ptr(self.zK), _ptr(self.zV), self.num_blocks)

    def tensors(self):
        return self.sK, self.sV, self.zK, self.zV

    def layer(self, l: int) -> PagedCache:
        return PagedCache(self.sK[l], self.sV[l], self.zK[l], self.zV[l])


def _layer_stride(t) -> int:
    return 0 if t is None else int(t.stride(0))


def lrkv_append_layers(dims: Dims, X, W_catT, slot_mapping, cache: LayeredCache, status=None, stream=None,
                       positions=None):
    """lrkv_append of the same slots in every layer: X [L, n, d], W_catT [L, N, d] -> the L layers' pools."""
    L, n = int(X.shape[0]), int(X.shape[1])
    st = LayerStrides(X=_layer_stride(X), W_catT=_layer_stride(W_catT), sK=_layer_stride(cache.sK),
                      sV=_layer_stride(cache.sV), zK=_layer_stride(cache.zK), zV=_layer_stride(cache.zV))
    c = cache.struct()
    rc = load().lrkv_append_layers(ctypes.byref(dims), L, ctypes.byref(st), _ptr(X), _ptr(W_catT), n,
                                   _ptr(slot_mapping), _ptr(positions), ctypes.byref(c), _ptr(status),
                                   _stream(stream))
    _check(rc, "lrkv_append_layers")


def lrkv_decode_layers(dims: Dims, q, BK, BV, cache: LayeredCache, block_table, seq_lens, out, workspace, status=None,
                       stream=None):
    """lrkv_decode of the same batch in every layer: q [L, B, H, d_h], B* [L, H, d_h, r] -> out [L, B, H, d_h];
    workspace of decode_workspace_bytes(dims, L * B) bytes."""
    L, B = int(q.shape[0]), int(q.shape[1])
    st = LayerStrides(q=_layer_stride(q), BK=_layer_stride(BK), BV=_layer_stride(BV), out=_layer_stride(out),
                      sK=_layer_stride(cache.sK), sV=_layer_stride(cache.sV), zK=_layer_stride(cache.zK),
                      zV=_layer_stride(cache.zV))
    c = cache.struct()
    rc = load().lrkv_decode_layers(ctypes.byref(dims), L, ctypes.byref(st), _ptr(q), _ptr(BK), _ptr(BV),
                                   ctypes.byref(c), _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens), B,
                                   _ptr(out), _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                   _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_layers")


_page_bytes: dict[tuple, int] = {}


class QuantCache:
    """One layer's quantised rows: uint8 [num_blocks, 64, quant_row_bytes(dims)]."""

    def __init__(self, rows):
        self.rows = rows
        self.num_blocks = int(rows.shape[0])

    @classmethod
    def empty(cls, dims: Dims, num_blocks: int, device="cuda"):
        return cls(torch.empty((num_blocks, 64, quant_row_bytes(dims)), dtype=torch.uint8, device=device))

    def struct(self, dims: Dims) -> QuantCacheStruct:
        # (the row's width by dims, so that a decode step need not ask the library for it)
        key = (dims.H, dims.d_h, dims.r, dims.d_rope, dims.block_size)
        page = _page_bytes.get(key)
        if page is None:
            page = quant_block_bytes(dims)
            if page:  # (0: dims that the call will refuse, perhaps for what is not in the key)
                _page_bytes[key] = page
        rows = self.rows
        if page and (rows.numel() != self.num_blocks * page or rows.dtype is not torch.uint8 or
                     not rows.is_contiguous()):
            raise ValueError(f"quantised rows {tuple(rows.shape)} of {rows.dtype}, strides {rows.stride()}: expected "
                             f"contiguous uint8 [num_blocks, 64, {quant_row_bytes(dims)}] for these dims")
        return QuantCacheStruct(_ptr(rows), self.num_blocks)


def quant_row_bytes(dims: Dims) -> int:
    return int(load().lrkv_quant_row_bytes(ctypes.byref(dims)))


def quant_block_bytes(dims: Dims) -> int:
    return int(load().lrkv_quant_block_bytes(ctypes.byref(dims)))


def decode_quant_workspace_bytes(dims: Dims, batch: int) -> int:
    return int(load().lrkv_decode_quant_workspace_bytes(ctypes.byref(dims), batch))


def decode_shared_workspace_bytes(dims: Dims, batch: int, max_prefix_blocks: int) -> int:
    return int(load().lrkv_decode_shared_workspace_bytes(ctypes.byref(dims), batch, max_prefix_blocks))


def lrkv_cache_quantize(dims: Dims, cache: PagedCache, bf16_slots, qcache: QuantCache, quant_slots, status=None,
                        stream=None):
    """Rows bf16_slots [n] of the bf16 pools -> rows quant_slots [n] of the quantised cache."""
    c, qc = cache.struct(), qcache.struct(dims)
    rc = load().lrkv_cache_quantize(ctypes.byref(dims), _same_length(bf16_slots, quant_slots), ctypes.byref(c),
                                    _ptr(bf16_slots), ctypes.byref(qc), _ptr(quant_slots), _ptr(status),
                                    _stream(stream))
    _check(rc, "lrkv_cache_quantize")


def lrkv_cache_dequantize(dims: Dims, qcache: QuantCache, quant_slots, cache: PagedCache, bf16_slots, status=None,
                          stream=None):
    """Rows quant_slots [n] of the quantised cache -> rows bf16_slots [n] of the bf16 pools (exact)."""
    c, qc = cache.struct(), qcache.struct(dims)
    rc = load().lrkv_cache_dequantize(ctypes.byref(dims), _same_length(bf16_slots, quant_slots), ctypes.byref(qc),
                                      _ptr(quant_slots), ctypes.byref(c), _ptr(bf16_slots), _ptr(status),
                                      _stream(stream))
    _check(rc, "lrkv_cache_dequantize")


def _same_length(a, b) -> int:
    n, m = a.shape[0], b.shape[0]
    if n != m:
        raise ValueError(f"slot arrays of {n} and {m} rows")
    return n


def lrkv_decode_quant(dims: Dims, q, BK, BV, qcache: QuantCache, block_table, seq_lens, out, workspace, status=None,
                      stream=None):
    """lrkv_decode over quantised rows: q [B, H, d_h] -> out [B, H, d_h]."""
    qc = qcache.struct(dims)
    rc = load().lrkv_decode_quant(ctypes.byref(dims), _ptr(q), _ptr(BK), _ptr(BV), ctypes.byref(qc),
                                  _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0],
                                  _ptr(out), _ptr(workspace), workspace.nbytes,
                                  _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_quant")


def lrkv_decode_quant_partials(dims: Dims, q, BK, qcache: QuantCache, block_table, seq_lens, partials, workspace,
                               status=None, stream=None):
    """lrkv_decode_partials over quantised rows: -> partials [B, H, d_h + r + 2] fp32."""
    qc = qcache.struct(dims)
    rc = load().lrkv_decode_quant_partials(ctypes.byref(dims), _ptr(q), _ptr(BK), ctypes.byref(qc),
                                           _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
                                           q.shape[0], _ptr(partials), _ptr(workspace),
                                           workspace.nbytes, _ptr(status),
                                           _stream(stream))
    _check(rc, "lrkv_decode_quant_partials")


def lrkv_decode_shared(dims: Dims, q, BK, BV, cache: PagedCache, prefix_blocks, prefix_len, block_table, seq_lens, out,
                       workspace, status=None, stream=None):
    """Decode of a batch that shares a prefix: prefix_blocks [max_prefix_blocks], prefix_len [1]; the sequences' own
    tokens in block_table, seq_lens (0 allowed): q [B, H, d_h] -> out [B, H, d_h]."""
    c = cache.struct()
    rc = load().lrkv_decode_shared(ctypes.byref(dims), _ptr(q), _ptr(BK), _ptr(BV), ctypes.byref(c),
                                   _ptr(prefix_blocks), prefix_blocks.shape[0], _ptr(prefix_len),
                                   _ptr(block_table), block_table.shape[1], _ptr(seq_lens), q.shape[0],
                                   _ptr(out), _ptr(workspace), workspace.nbytes,
                                   _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_shared")


def lrkv_prefix_partials(dims: Dims, q, BK, cache: PagedCache, prefix_blocks, prefix_len, partials, workspace,
                         status=None, stream=None):
    """Decode partials of the whole batch over the shared prefix: -> partials [B, H, d_h + r + 2] fp32."""
    c = cache.struct()
    rc = load().lrkv_prefix_partials(ctypes.byref(dims), _ptr(q), _ptr(BK), ctypes.byref(c), _ptr(prefix_blocks),
                                     prefix_blocks.shape[0], _ptr(prefix_len), q.shape[0], _ptr(partials),
                                     _ptr(workspace), workspace.nbytes,
                                     _ptr(status), _stream(stream))
    _check(rc, "lrkv_prefix_partials")


def decode_tree_workspace_bytes(dims: Dims, batch: int, T: int) -> int:
    return int(load().lrkv_decode_tree_workspace_bytes(ctypes.byref(dims), batch, T))


_I32, _I64 = torch.int32, torch.int64


def _words(t, n: int):
    """Pointer of n contiguous 32-bit words (a pointer or None: as it is)."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not _I32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{tuple(t.shape)} of {t.dtype}, strides {t.stride()}: expected contiguous int32 [{n}]")
    return t.data_ptr()


def lrkv_decode_tree(dims: Dims, q, BK, BV, cache: PagedCache, block_table, seq_lens, tree_mask, tree_lens, out,
                     workspace, status=None, stream=None):
    """Drafted tokens over the cache: q [B, T, H, d_h + d_rope] -> out [B, T, H, d_h]; tree_mask [B, T] int64 bit sets
    of the drafted tokens seen (None: a chain), tree_lens [B] int32 drafted tokens of each sequence (None: T)."""
    c = cache.struct()
    B, T = q.shape[:2]
    if tree_mask is not None and ((tree_mask.dtype is not _I64 and tree_mask.dtype is not torch.uint64) or
                                  tree_mask.shape != (B, T) or not tree_mask.is_contiguous()):
        raise ValueError(f"tree_mask {tuple(tree_mask.shape)} of {tree_mask.dtype}, strides {tree_mask.stride()}: "
                         f"expected contiguous 64-bit words [{B}, {T}]")
    rows, width = block_table.shape
    if block_table.dtype is not _I32 or rows != B or not block_table.is_contiguous():
        raise ValueError(f"block table {tuple(block_table.shape)} of {block_table.dtype}, strides "
                         f"{block_table.stride()}: expected contiguous int32 [{B}, ...]")
    rc = load().lrkv_decode_tree(ctypes.byref(dims), q.data_ptr(), _ptr(BK), _ptr(BV), ctypes.byref(c),
                                 block_table.data_ptr(), width, _words(seq_lens, B), _ptr(tree_mask),
                                 _words(tree_lens, B), B, T, _ptr(out), workspace.data_ptr(), workspace.nbytes,
                                 _ptr(status), _stream(stream))
    _check(rc, "lrkv_decode_tree")


_ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "parts": 2}
_ROPE_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def rope_plan(d_rot: int, layout: str = "interleaved", base: float = 10000.0, scaling: str = "none",
              factor: float = 1.0, original_len: float = 0.0, low: float = 1.0, high: float = 32.0,
              magnitude: float = 1.0) -> RopePlan:
    """Speeds of a rotation of d_rot values per head (lrkv_rope_make_plan); made once, kept by the caller."""
    spec = RopeSpec(d_rot, _ROPE_LAYOUTS[layout], _ROPE_SCALINGS[scaling], 0, base, factor, original_len, low, high,
                    magnitude)
    plan = RopePlan()
    _check(load().lrkv_rope_make_plan(ctypes.byref(spec), ctypes.byref(plan)), "lrkv_rope_make_plan")
    return plan


def lrkv_rope(plan: RopePlan, x, y, positions, begin: int = 0, x_rows=None, y_rows=None, transpose: bool = False,
              status=None, stream=None):
    """y = x with values [begin, begin + plan.d_rot) of every head rotated at positions [n] (int32): x, y
    [rows, heads, width] of bf16 or fp32 (y is x: in place); x_rows, y_rows [n] int32 pick rows."""
    n = positions.shape[0]
    xs, xt = x.shape, x.stride()
    ys, yt = (xs, xt) if y is x else (y.shape, y.stride())
    kind = _ROPE_TYPES.get(x.dtype)
    if (kind is None or y.dtype is not x.dtype or len(xs) != 3 or len(ys) != 3 or xs[1] != ys[1] or xs[2] != ys[2] or
            xt[2] != 1 or yt[2] != 1):
        raise ValueError(f"x {tuple(xs)} of {x.dtype}, strides {xt}; y {tuple(ys)} of {y.dtype}, strides {yt}: expected "
                         "[rows, heads, width] of equal heads and widths, bfloat16 or float32, last stride 1")
    xr = RowsStruct(x.data_ptr(), xs[0], xt[0], xt[1], _words(x_rows, n))
    yr = RowsStruct(y.data_ptr(), ys[0], yt[0], yt[1], _words(y_rows, n))
    rc = load().lrkv_rope(ctypes.byref(plan), kind, n, xs[1], xs[2], begin, ctypes.byref(xr), ctypes.byref(yr),
                          _words(positions, n), 1 if transpose else 0, _ptr(status), _stream(stream))
    _check(rc, "lrkv_rope")


class Pools:
    """Pools whose rows move together (lrkv_pools): made once from a cache and kept (it keeps the tensors)."""

    def __init__(self, tensors):
        """tensors: [layers, num_blocks, 64, ...] each, a layer contiguous."""
        self.tensors = tuple(tensors)
        s = self.c = PoolsStruct()
        first = self.tensors[0]
        s.num_pools, s.num_layers, s.num_blocks = len(self.tensors), first.shape[0], first.shape[1]
        if not 1 <= len(self.tensors) <= 4:
            raise ValueError(f"{len(self.tensors)} pools (1 to 4)")
        for i, t in enumerate(self.tensors):
            if t.dim() < 4 or t.shape[:3] != (first.shape[0], first.shape[1], 64) or not t[0].is_contiguous():
                raise ValueError(f"pool {tuple(t.shape)}, strides {t.stride()}: expected [layers, num_blocks, 64, ...], "
                                 "each layer contiguous, alike in all pools")
            s.base[i] = _ptr(t)
            s.row_bytes[i] = t[0, 0, 0].numel() * t.element_size()
            s.layer_bytes[i] = t.stride(0) * t.element_size()

    @classmethod
    def of(cls, cache):
        """Of a PagedCache, a LayeredCache, a QuantCache, or a pool tensor [num_blocks, 64, ...]."""
        if isinstance(cache, LayeredCache):
            return cls(cache.tensors())
        if isinstance(cache, PagedCache):
            return cls(t.unsqueeze(0) for t in cache.tensors())
        return cls([(cache.rows if isinstance(cache, QuantCache) else cache).unsqueeze(0)])


def _page_table(refs, block_table, seq_lens):
    """Checks of what the page calls write; the table's shape."""
    if (refs.dtype is not _I32 or block_table.dtype is not _I32 or seq_lens.dtype is not _I32 or
            not refs.is_contiguous() or not block_table.is_contiguous() or not seq_lens.is_contiguous()):
        raise ValueError(f"counts or paths of {refs.dtype}, block table of {block_table.dtype}, lengths of "
                         f"{seq_lens.dtype}: expected contiguous int32")
    shape = block_table.shape
    if shape[0] != seq_lens.shape[0]:
        raise ValueError(f"block table of {shape[0]} sequences, {seq_lens.shape[0]} lengths")
    return shape


def lrkv_pages_reserve(refs, block_table, seq_lens, new_tokens, status=None, stream=None):
    """Pages for new_tokens [B] more tokens of every sequence, from the pages with count 0 in refs [num_blocks]."""
    B, width = _page_table(refs, block_table, seq_lens)
    rc = load().lrkv_pages_reserve(refs.shape[0], _ptr(refs), _ptr(block_table), width, _ptr(seq_lens),
                                   _words(new_tokens, B), B, _ptr(status), _stream(stream))
    _check(rc, "lrkv_pages_reserve")


def lrkv_pages_fork(pools: Pools, refs, block_table, seq_lens, parents, children, status=None, stream=None):
    """Sequences children [n] become copies of sequences parents [n], sharing their full pages."""
    B, width = _page_table(refs, block_table, seq_lens)
    if refs.shape[0] != pools.c.num_blocks:
        raise ValueError(f"{refs.shape[0]} counts for {pools.c.num_blocks} pages")
    n = parents.shape[0]
    rc = load().lrkv_pages_fork(ctypes.byref(pools.c), _ptr(refs), _ptr(block_table), width, _ptr(seq_lens),
                                B, _words(parents, n), _words(children, n), n, _ptr(status), _stream(stream))
    _check(rc, "lrkv_pages_fork")


def lrkv_pages_free(refs, block_table, seq_lens, seqs, keep_lens=None, status=None, stream=None):
    """Sequences seqs [n] give back their pages behind keep_lens [B] tokens (None: all)."""
    B, width = _page_table(refs, block_table, seq_lens)
    n = seqs.shape[0]
    rc = load().lrkv_pages_free(refs.shape[0], _ptr(refs), _ptr(block_table), width, _ptr(seq_lens), B,
                                _words(seqs, n), n, _words(keep_lens, B), _ptr(status), _stream(stream))
    _check(rc, "lrkv_pages_free")


def lrkv_pages_copy(src: Pools, src_pages, dst: Pools, dst_pages, status=None, stream=None):
    """Pages src_pages [n] of src -> pages dst_pages [n] of dst, in all pools and layers."""
    n = src_pages.shape[0]
    rc = load().lrkv_pages_copy(ctypes.byref(src.c), _words(src_pages, n), ctypes.byref(dst.c), _words(dst_pages, n), n,
                                _ptr(status), _stream(stream))
    _check(rc, "lrkv_pages_copy")


def lrkv_cache_compact(pools: Pools, block_table, seq_lens, path, path_lens, new_lens=None, status=None, stream=None):
    """Rows seq_lens[b] + path[b, i] -> seq_lens[b] + i, i < path_lens[b]; new_lens = seq_lens + path_lens (None: in
    place)."""
    B, width = _page_table(path, block_table, seq_lens)
    rows, max_path = path.shape
    if rows != B:
        raise ValueError(f"paths of {rows} sequences, {B} lengths")
    rc = load().lrkv_cache_compact(ctypes.byref(pools.c), _ptr(block_table), width, _ptr(seq_lens), B,
                                   _ptr(path), _words(path_lens, B), max_path, _words(new_lens, B), _ptr(status),
                                   _stream(stream))
    _check(rc, "lrkv_cache_compact")


def lrkv_prefill(dims: Dims, q, BK, BV, cache: PagedCache, block_table, q_start, out, workspace=None, status=None,
                 stream=None):
    """Causal chunked prefill: q [B, Tq, H, d_h] at positions q_start[b] + i -> out [B, Tq, H, d_h]."""
    B, Tq = int(q.shape[0]), int(q.shape[1])
    c = cache.struct()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().lrkv_prefill(ctypes.byref(dims), _ptr(q), _ptr(BK), _ptr(BV), ctypes.byref(c), _ptr(block_table),
                             int(block_table.shape[1]), _ptr(q_start), B, Tq, _ptr(out), _ptr(workspace), ws_bytes,
                             _ptr(status), _stream(stream))
    _check(rc, "lrkv_prefill")


def lrkv_prefill_fused(dims: Dims, q, q_tilde, cache: PagedCache, block_table, q_start, out, status=None, stream=None):
    """Causal prefill with absorbed weights: q [B, Tq, H, d_h], q~ [B, Tq, H, r] -> out [B, Tq, H, d_h + r]."""
    B, Tq = int(q.shape[0]), int(q.shape[1])
    c = cache.struct()
    rc = load().lrkv_prefill_fused(ctypes.byref(dims), _ptr(q), _ptr(q_tilde), ctypes.byref(c), _ptr(block_table),
                                   int(block_table.shape[1]), _ptr(q_start), B, Tq, _ptr(out), _ptr(status),
                                   _stream(stream))
    _check(rc, "lrkv_prefill_fused")


def train_workspace_bytes(dims: Dims, n_tok: int) -> int:
    return int(load().lrkv_train_workspace_bytes(ctypes.byref(dims), n_tok))


def lrkv_train_forward(dims: Dims, X, W_T, B, Y, K, status=None, stream=None):
    """Expanded projection: Y = X W_T^T = [S | R] ([n, d_h + H r]) and K = S + R_h B_h^T ([n, H, d_h])."""
    rc = load().lrkv_train_forward(ctypes.byref(dims), _ptr(X), _ptr(W_T), _ptr(B), int(X.shape[0]), _ptr(Y),
                                   _ptr(K), _ptr(status), _stream(stream))
    _check(rc, "lrkv_train_forward")


def lrkv_train_backward(dims: Dims, X, W_T, B, Y, dK, dX, dW_T, dB, workspace, status=None, stream=None):
    """Gradients through K_h = X (W_shared + U_h B_h^T): dX [n, d], dW_T [d_h + H r, d], dB [H, d_h, r]."""
    rc = load().lrkv_train_backward(ctypes.byref(dims), _ptr(X), _ptr(W_T), _ptr(B), _ptr(Y), _ptr(dK),
                                    int(X.shape[0]), _ptr(dX), _ptr(dW_T), _ptr(dB), _ptr(workspace),
                                    int(workspace.numel() * workspace.element_size()), _ptr(status),
                                    _stream(stream))
    _check(rc, "lrkv_train_backward")


def pack_side_t(Ws, U) -> torch.Tensor:
    """W_T [d_h + H r, d] of one projection from W_shared [d, d_h] and U [H, d, r]."""
    H, d, r = U.shape
    return torch.cat([Ws.t(), U.permute(0, 2, 1).reshape(H * r, d)], dim=0).contiguous()


def mla_cache_block_bytes(dims: MlaDims) -> int:
    return int(load().lrkv_mla_cache_block_bytes(ctypes.byref(dims)))


def mla_decode_workspace_bytes(dims: MlaDims, batch: int) -> int:
    return int(load().lrkv_mla_decode_workspace_bytes(ctypes.byref(dims), batch))


def lrkv_mla_append(dims: MlaDims, X, W_T, slot_mapping, positions, kv, status=None, stream=None):
    """MLA cache rows [c | RoPE(k^R)] of X [n, d] into kv [num_blocks, 64, d_c + d_rope] at slot_mapping [n]."""
    rc = load().lrkv_mla_append(ctypes.byref(dims), _ptr(X), _ptr(W_T), int(X.shape[0]), _ptr(slot_mapping),
                                _ptr(positions), _ptr(kv), int(kv.shape[0]), _ptr(status), _stream(stream))
    _check(rc, "lrkv_mla_append")


def lrkv_mla_decode(dims: MlaDims, q, kv, block_table, seq_lens, out, workspace, status=None, stream=None):
    """Absorbed MLA decode: q [B, H, d_c + d_rope] -> out [B, H, d_c]."""
    rc = load().lrkv_mla_decode(ctypes.byref(dims), _ptr(q), _ptr(kv), int(kv.shape[0]), _ptr(block_table),
                                int(block_table.shape[1]), _ptr(seq_lens), int(q.shape[0]), _ptr(out),
                                _ptr(workspace), int(workspace.numel() * workspace.element_size()), _ptr(status),
                                _stream(stream))
    _check(rc, "lrkv_mla_decode")


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned device byte buffer (torch's allocator aligns to 512 B)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def pack_wcat_t(WsK, WsV, UK, UV, WKR=None) -> torch.Tensor:
    """W_cat^T [N, d] from W_shared^{K,V} [d, d_h], U^{K,V} [H, d, r] and the optional positional-key
    projection W^KR [d, d_rope] (column order of lrkv_append)."""
    H, d, r = UK.shape
    parts = [WsK.t()] + ([] if WKR is None else [WKR.t()])
    return torch.cat(parts + [WsV.t(), UK.permute(0, 2, 1).reshape(H * r, d),
                              UV.permute(0, 2, 1).reshape(H * r, d)], dim=0).contiguous()
