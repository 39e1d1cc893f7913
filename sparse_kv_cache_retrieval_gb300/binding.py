"""ctypes binding of libspc.so: the C entry points under the same names.

Marshalling only: tensors become device (or host) pointers, the stream
defaults to torch's current CUDA stream, a non-zero status raises SpcError.
Every computation runs in the library's CUDA kernels; if the library is
missing or cannot be loaded, the first call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspc.so")

SPC_OK = 0
STATUS_NAMES = {0: "SPC_OK", -1: "SPC_ERR_INVALID_ARG", -2: "SPC_ERR_SHAPE", -3: "SPC_ERR_CUDA",
                -4: "SPC_ERR_TIMEOUT", -5: "SPC_ERR_WORKSPACE", -6: "SPC_ERR_OVERFLOW"}

# struct layouts of include/spc.h (32 bytes each)
GATHER_VIEW_DTYPE = np.dtype([("host", "<u8"), ("slots", "<u8"), ("layer0", "<i4"),
                              ("n_layers", "<i4"), ("store_layer0", "<i4"), ("store_layers", "<i4")])
KV_VIEW_DTYPE = np.dtype([("k", "<u8"), ("v", "<u8"), ("rows", "<i8"), ("use_slots", "<i4"),
                          ("reserved", "<i4")])

_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
SIGNATURES = {
    "spc_status_string": (ctypes.c_char_p, [_I]),
    "spc_version": (_I, []),
    "spc_device_sm_count": (_I, []),
    "spc_score_select_workspace_size": (ctypes.c_size_t, [_I] * 7),
    "spc_score_select": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P,
                              _P, ctypes.c_size_t, _P]),
    "spc_score_select_stages": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P,
                                     _P, _P, ctypes.c_size_t, _P, _I]),
    "spc_elastic_diff": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "spc_gather_kv": (_I, [_P, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "spc_sparse_decode_attn_workspace_size": (ctypes.c_size_t, [_I] * 6),
    "spc_sparse_decode_attn": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P,
                                    ctypes.c_size_t, _P]),
    "spc_sparse_decode_attn_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float,
                                            _P, _P]),
    "spc_host_device_pointer": (_I, [_P, ctypes.POINTER(ctypes.c_void_p)]),
    "spc_stream_read": (_I, [_P, ctypes.c_size_t, _P, _I, _P]),
    "spc_copy": (_I, [_P, _P, ctypes.c_size_t, _P]),
    "spc_fill_slots": (_I, [_P, _I, _I, _P, _I, _I, _I, _I, _I, _P]),
    "spc_store_layer": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "spc_offload_thresholds": (_I, [_I, _I, _I, _I, _I, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]),
    "spc_batch_select_workspace_size": (ctypes.c_size_t, [_I] * 3),
    "spc_batch_select": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, ctypes.c_size_t, _P]),
    "spc_mla_score_select_workspace_size": (ctypes.c_size_t, [_I] * 4),
    "spc_mla_score_select": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P,
                                  ctypes.c_size_t, _P, _I]),
    "spc_mla_gather": (_I, [_P, _I, _I, _P, _P, _P, _I, _I, _I, _P]),
    "spc_block_map": (_I, [_P] * 9 + [_I] * 5 + [_P]),
    "spc_kv4_store": (_I, [_P, _P, ctypes.c_int64, ctypes.c_int64, _P, _P, _I, _I, _I, _I, _I, _P]),
    "spc_kv4_load": (_I, [_P, _P, _P, _P, ctypes.c_int64, ctypes.c_int64, _I, _I, _I, _I, _I, _P]),
    "spc_kv4_decode_attn_workspace_size": (ctypes.c_size_t, [_I] * 7),
    "spc_kv4_decode_attn": (_I, [_P] * 5 + [_I] * 8 + [ctypes.c_float, _P, _P, ctypes.c_size_t, _P]),
    "spc_prompt_attn_workspace_size": (ctypes.c_size_t, [_I] * 5),
    "spc_prompt_attn": (_I, [_P] * 4 + [_I] * 5 + [ctypes.c_int64] * 3 + [ctypes.c_float, _P, _P, ctypes.c_size_t,
                                                                         _P]),
    "spc_kv4_chunk_attn_workspace_size": (ctypes.c_size_t, [_I] * 5),
    "spc_kv4_chunk_attn": (_I, [_P] * 5 + [_I] * 8 + [ctypes.c_int64, ctypes.c_float, _P, _P, _P, ctypes.c_size_t, _P]),
    "spc_kv4_attn_mass_workspace_size": (ctypes.c_size_t, [_I] * 5),
    "spc_kv4_attn_mass": (_I, [_P] * 8 + [_I] * 9 + [ctypes.c_int64, ctypes.c_float, ctypes.c_float, _P, ctypes.c_size_t,
                                                    _P]),
    "spc_kv4_evict": (_I, [_P] * 9 + [_I] * 10 + [_P]),
    "spc_mla_decode_attn_workspace_size": (ctypes.c_size_t, [_I] * 3),
    "spc_mla_decode_attn": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, ctypes.c_float, _P, _P, ctypes.c_size_t,
                                 _P]),
}


class SpcError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}: "
                         f"{lib().spc_status_string(status).decode()}")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(handle, name)
            f.restype = res
            f.argtypes = args
        _lib = handle
    return _lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return t.data_ptr()
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(t)}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int) -> None:
    if status != SPC_OK:
        raise SpcError(fn, status)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# ------------------------------------------------------------------ entry points
def spc_score_select_workspace_size(B, H, n_q, n_kv, d, cap, budget) -> int:
    return int(lib().spc_score_select_workspace_size(B, H, n_q, n_kv, d, cap, budget))


def spc_score_select(x, Wq, Wk, K_dlm, len, append, B, H, n_q, n_kv, d, cap, budget, n_sink,
                     n_recent, q_out, scores_out, selected, workspace, workspace_bytes=None,
                     stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    _check("spc_score_select", lib().spc_score_select(
        _ptr(x), _ptr(Wq), _ptr(Wk), _ptr(K_dlm), _ptr(len), int(append), B, H, n_q, n_kv, d, cap,
        budget, n_sink, n_recent, _ptr(q_out), _ptr(scores_out), _ptr(selected), _ptr(workspace),
        workspace_bytes, _stream(stream)))


SPC_STAGE_PROJECT, SPC_STAGE_SCAN, SPC_STAGE_SELECT = 1, 2, 4


def spc_score_select_stages(x, Wq, Wk, K_dlm, len, append, B, H, n_q, n_kv, d, cap, budget, n_sink,
                            n_recent, q_out, scores_out, selected, workspace, workspace_bytes=None,
                            stream=None, stages=7) -> None:
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    _check("spc_score_select_stages", lib().spc_score_select_stages(
        _ptr(x), _ptr(Wq), _ptr(Wk), _ptr(K_dlm), _ptr(len), int(append), B, H, n_q, n_kv, d, cap,
        budget, n_sink, n_recent, _ptr(q_out), _ptr(scores_out), _ptr(selected), _ptr(workspace),
        workspace_bytes, _stream(stream), int(stages)))


def spc_elastic_diff(selected, slot_pos_prev, slot_pos_next, load_slot, load_pos, n_load, B, n_kv,
                     budget, cap, stream=None) -> None:
    _check("spc_elastic_diff", lib().spc_elastic_diff(
        _ptr(selected), _ptr(slot_pos_prev), _ptr(slot_pos_next), _ptr(load_slot), _ptr(load_pos),
        _ptr(n_load), B, n_kv, budget, cap, _stream(stream)))


def spc_gather_kv(views, layer_lo, layer_hi, load_slot, load_pos, n_load, B, n_kv, d, cap, budget,
                  stream=None) -> None:
    _check("spc_gather_kv", lib().spc_gather_kv(
        _ptr(views), layer_lo, layer_hi, _ptr(load_slot), _ptr(load_pos), _ptr(n_load), B, n_kv, d,
        cap, budget, _stream(stream)))


def spc_sparse_decode_attn_workspace_size(n_layers, B, n_q, n_kv, d, budget) -> int:
    return int(lib().spc_sparse_decode_attn_workspace_size(n_layers, B, n_q, n_kv, d, budget))


def spc_sparse_decode_attn(q, views, selected, slot_pos, n_layers, B, n_q, n_kv, d, budget, scale,
                           out, workspace, workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    _check("spc_sparse_decode_attn", lib().spc_sparse_decode_attn(
        _ptr(q), _ptr(views), _ptr(selected), _ptr(slot_pos), n_layers, B, n_q, n_kv, d, budget,
        float(scale), _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)))


SPC_ATTN_NOALLOC_SCRATCH_BYTES = 8 << 20


def spc_sparse_decode_attn_noalloc(q, views, selected, slot_pos, n_layers, B, n_q, n_kv, d, budget,
                                   scale, out, stream=None) -> None:
    """spc_sparse_decode_attn with the library's fixed scratch area instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _check("spc_sparse_decode_attn_noalloc", lib().spc_sparse_decode_attn_noalloc(
        _ptr(q), _ptr(views), _ptr(selected), _ptr(slot_pos), n_layers, B, n_q, n_kv, d, budget,
        float(scale), _ptr(out), _stream(stream)))


def spc_host_device_pointer(host) -> int:
    out = ctypes.c_void_p()
    _check("spc_host_device_pointer", lib().spc_host_device_pointer(_ptr(host), ctypes.byref(out)))
    return int(out.value)


def spc_stream_read(src, nbytes, sink, n_blocks, stream=None) -> None:
    _check("spc_stream_read", lib().spc_stream_read(_ptr(src), nbytes, _ptr(sink), n_blocks,
                                                    _stream(stream)))


def spc_copy(dst, src, nbytes, stream=None) -> None:
    """Kernel copy between device memory and device-visible host addresses."""
    _check("spc_copy", lib().spc_copy(_ptr(dst), _ptr(src), int(nbytes), _stream(stream)))


def spc_fill_slots(views, layer_lo, layer_hi, slot_pos, B, n_kv, d, cap, budget, stream=None) -> None:
    _check("spc_fill_slots", lib().spc_fill_slots(_ptr(views), layer_lo, layer_hi, _ptr(slot_pos), B,
                                                  n_kv, d, cap, budget, _stream(stream)))


def spc_store_layer(store, src, n_kv, d, cap, rows, store_layers, layer, stream=None) -> None:
    _check("spc_store_layer", lib().spc_store_layer(_ptr(store), _ptr(src), n_kv, d, cap, rows, store_layers,
                                                    layer, _stream(stream)))


def spc_offload_thresholds(n_layers, n_kv, d, B, budget, kv_bytes) -> list:
    """Host-side memory model: n_layers + 1 context-length thresholds (the
    last one is INT64_MAX)."""
    out = (ctypes.c_int64 * (n_layers + 1))()
    _check("spc_offload_thresholds", lib().spc_offload_thresholds(n_layers, n_kv, d, B, budget,
                                                                  int(kv_bytes), out))
    return [int(v) for v in out]


def spc_batch_select_workspace_size(B, cap, budget) -> int:
    return int(lib().spc_batch_select_workspace_size(B, cap, budget))


def spc_batch_select(scores, len, B, n_kv, cap, budget, n_sink, n_recent, selected, workspace, workspace_bytes=None,
                     stream=None) -> None:
    """Batch-level selection: one Top-K per request from the max over groups,
    copied to every KV head."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    _check("spc_batch_select", lib().spc_batch_select(
        _ptr(scores), _ptr(len), B, n_kv, cap, budget, n_sink, n_recent, _ptr(selected), _ptr(workspace),
        workspace_bytes, _stream(stream)))


# ------------------------------------------------------------------ MLA variant
SPC_MLA_LATENT, SPC_MLA_ROPE, SPC_MLA_NOPE, SPC_MLA_V, SPC_MLA_HEADS = 512, 64, 128, 128, 16


def spc_mla_score_select_workspace_size(B, H, cap, budget) -> int:
    return int(lib().spc_mla_score_select_workspace_size(B, H, cap, budget))


def spc_mla_score_select(x, Wq, Wuk, Wdkv, C_dlm, len, append, B, H, cap, budget, n_sink, n_recent,
                         scores_out, selected, workspace, workspace_bytes=None, stream=None, stages=7) -> None:
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    _check("spc_mla_score_select", lib().spc_mla_score_select(
        _ptr(x), _ptr(Wq), _ptr(Wuk), _ptr(Wdkv), _ptr(C_dlm), _ptr(len), int(append), B, H, cap, budget,
        n_sink, n_recent, _ptr(scores_out), _ptr(selected), _ptr(workspace), workspace_bytes, _stream(stream),
        int(stages)))


def spc_mla_gather(views, layer_lo, layer_hi, load_slot, load_pos, n_load, B, cap, budget, stream=None) -> None:
    _check("spc_mla_gather", lib().spc_mla_gather(
        _ptr(views), layer_lo, layer_hi, _ptr(load_slot), _ptr(load_pos), _ptr(n_load), B, cap, budget,
        _stream(stream)))


def spc_mla_decode_attn_workspace_size(n_layers, B, budget) -> int:
    return int(lib().spc_mla_decode_attn_workspace_size(n_layers, B, budget))


def spc_mla_decode_attn(q, Wuk, Wuv, views, selected, slot_pos, n_layers, B, budget, scale, out, workspace,
                        workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    _check("spc_mla_decode_attn", lib().spc_mla_decode_attn(
        _ptr(q), _ptr(Wuk), _ptr(Wuv), _ptr(views), _ptr(selected), _ptr(slot_pos), n_layers, B, budget,
        float(scale), _ptr(out), _ptr(workspace), workspace_bytes, _stream(stream)))


# ------------------------------------------------------------------ paged 4-bit cache
SPC_KV4_RECORD, SPC_KV4_GROUP = 144, 16

# accepted dtypes, filled in by _device() (torch is imported on first use)
_BF16, _I32, _BYTES, _F32 = set(), set(), set(), set()


_torch = None


def _device():
    """Index of the current CUDA device (-2, no tensor's, before CUDA is up)."""
    global _torch
    if _torch is None:
        import torch
        _BF16.update((torch.bfloat16, torch.int16, torch.uint16))
        _BYTES.update((torch.uint8, torch.int8))
        _I32.add(torch.int32)
        _F32.add(torch.float32)
        _torch = torch
    return _torch.cuda.current_device() if _torch.cuda.is_initialized() else -2


def _raw_stream(stream, dev):
    if stream is None:
        # the handle alone: torch.cuda.current_stream builds a Stream object, 1-2 us a call
        return _torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dev(name, t, dtypes, numel, dev):
    """Pointer of a contiguous tensor of at least `numel` elements on device
    `dev` (an int is taken as a device address, None stays None)."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype in dtypes and t.numel() >= numel and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {', '.join(sorted(map(str, dtypes)))}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, {numel} needed")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    raise _wrong_device(name, t, dev)


def _wrong_device(name, t, dev):
    return ValueError(f"{name}: tensor is on {t.device}, expected " +
                      (f"the current device cuda:{dev}" if dev >= 0 else "a CUDA device"))


def _rows(name, t, T, n, d, stride, dev):
    """(pointer, row stride in elements) of bf16 rows [T][n][d] whose rows may
    lie `stride` elements apart."""
    if t is None or isinstance(t, int):
        return t, n * d if stride is None else int(stride)
    if t.dtype not in _BF16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected bf16 values or bit patterns")
    shape = t.shape
    if len(shape) != 3 or shape[0] < T or shape[1] != n or shape[2] != d:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [{T}][{n}][{d}]")
    s0, s1, s2 = t.stride()
    # a dimension of one element may carry any stride, and a tensor of none has none
    if shape[0] and ((s2 != 1 and d > 1) or (s1 != d and n > 1)):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if shape[0] <= 1:
        s0 = n * d
    if stride is not None and stride != s0:
        raise ValueError(f"{name}: stride {stride} given for a tensor of row stride {s0}")
    if t.get_device() != dev:
        raise _wrong_device(name, t, dev)
    return t.data_ptr(), s0


def spc_block_map(len, len_next, block_table, free_list, n_free, n_free_next, cu_new, slot_map, status, B, max_blocks,
                  block_size, num_blocks, n_slots, stream=None) -> None:
    """Block tables, free stack and slot map of the requests' next lengths."""
    dev = _device()
    _check("spc_block_map", lib().spc_block_map(
        _dev("len", len, _I32, B, dev), _dev("len_next", len_next, _I32, B, dev),
        _dev("block_table", block_table, _I32, B * max_blocks, dev), _dev("free_list", free_list, _I32, num_blocks, dev),
        _dev("n_free", n_free, _I32, 1, dev), _dev("n_free_next", n_free_next, _I32, 1, dev),
        _dev("cu_new", cu_new, _I32, B + 1, dev), _dev("slot_map", slot_map, _I32, n_slots, dev),
        _dev("status", status, _I32, 1, dev), B, max_blocks, block_size, num_blocks, n_slots, _raw_stream(stream, dev)))


def spc_kv4_store(k, v, slot_map, cache, T, n_kv, d, num_blocks, block_size, k_stride=None, v_stride=None,
                  stream=None) -> None:
    """Rows of K and V into the slots of the 4-bit cache. The row strides are
    the tensors' own; they are given only with plain addresses."""
    dev = _device()
    k, k_stride = _rows("k", k, T, n_kv, d, k_stride, dev)
    v, v_stride = _rows("v", v, T, n_kv, d, v_stride, dev)
    _check("spc_kv4_store", lib().spc_kv4_store(
        k, v, k_stride, v_stride, _dev("slot_map", slot_map, _I32, T, dev),
        _dev("cache", cache, _BYTES, num_blocks * n_kv * block_size * SPC_KV4_RECORD, dev), T, n_kv, d, num_blocks,
        block_size, _raw_stream(stream, dev)))


def spc_kv4_load(cache, slot_map, k, v, T, n_kv, d, num_blocks, block_size, k_stride=None, v_stride=None,
                 stream=None) -> None:
    """Rows of the 4-bit cache's slots as bf16 (exact)."""
    dev = _device()
    k, k_stride = _rows("k", k, T, n_kv, d, k_stride, dev)
    v, v_stride = _rows("v", v, T, n_kv, d, v_stride, dev)
    _check("spc_kv4_load", lib().spc_kv4_load(
        _dev("cache", cache, _BYTES, num_blocks * n_kv * block_size * SPC_KV4_RECORD, dev),
        _dev("slot_map", slot_map, _I32, T, dev), k, v, k_stride, v_stride, T, n_kv, d, num_blocks, block_size,
        _raw_stream(stream, dev)))


def spc_kv4_decode_attn_workspace_size(B, n_q, n_kv, d, max_blocks, block_size, budget) -> int:
    return int(lib().spc_kv4_decode_attn_workspace_size(B, n_q, n_kv, d, max_blocks, block_size, budget))


def spc_kv4_decode_attn(q, cache, block_table, len, selected, B, n_q, n_kv, d, num_blocks, block_size, max_blocks,
                        budget, scale, out, workspace, workspace_bytes=None, stream=None) -> None:
    """Decode attention over the paged 4-bit cache: the whole context, or
    (selected, budget) the positions kept per KV head."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    dev = _device()
    _check("spc_kv4_decode_attn", lib().spc_kv4_decode_attn(
        _dev("q", q, _BF16, B * n_q * d, dev),
        _dev("cache", cache, _BYTES, num_blocks * n_kv * block_size * SPC_KV4_RECORD, dev),
        _dev("block_table", block_table, _I32, B * max_blocks, dev), _dev("len", len, _I32, B, dev),
        _dev("selected", selected, _I32, B * n_kv * budget, dev), B, n_q, n_kv, d, num_blocks, block_size, max_blocks,
        budget, float(scale), _dev("out", out, _BF16, B * n_q * d, dev), _dev("workspace", workspace, _BYTES, workspace_bytes, dev),
        workspace_bytes, _raw_stream(stream, dev)))


def spc_prompt_attn_workspace_size(T, B, n_q, n_kv, d) -> int:
    return int(lib().spc_prompt_attn_workspace_size(T, B, n_q, n_kv, d))


def spc_prompt_attn(q, k, v, cu_seqlens, T, B, n_q, n_kv, d, scale, out, workspace, workspace_bytes=None,
                    q_stride=None, k_stride=None, v_stride=None, stream=None) -> None:
    """Causal attention over B packed prompts. The row strides are the
    tensors' own; they are given only with plain addresses."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    dev = _device()
    q, q_stride = _rows("q", q, T, n_q, d, q_stride, dev)
    k, k_stride = _rows("k", k, T, n_kv, d, k_stride, dev)
    v, v_stride = _rows("v", v, T, n_kv, d, v_stride, dev)
    _check("spc_prompt_attn", lib().spc_prompt_attn(
        q, k, v, _dev("cu_seqlens", cu_seqlens, _I32, B + 1, dev), T, B, n_q, n_kv, d, q_stride, k_stride, v_stride,
        float(scale), _dev("out", out, _BF16, T * n_q * d, dev),
        _dev("workspace", workspace, _BYTES, workspace_bytes, dev), workspace_bytes, _raw_stream(stream, dev)))


def spc_kv4_chunk_attn_workspace_size(T, B, n_q, n_kv, d) -> int:
    return int(lib().spc_kv4_chunk_attn_workspace_size(T, B, n_q, n_kv, d))


def spc_kv4_chunk_attn(q, cache, block_table, len, cu_seqlens, T, B, n_q, n_kv, d, num_blocks, block_size, max_blocks,
                       scale, out, lse, workspace, workspace_bytes=None, q_stride=None, stream=None) -> None:
    """Attention of B requests' new tokens, packed, over the paged 4-bit cache
    that holds them already, and (unless lse is None) the rows' log-sum-exp.
    The row stride is q's own; it is given only with a plain address."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    dev = _device()
    q, q_stride = _rows("q", q, T, n_q, d, q_stride, dev)
    _check("spc_kv4_chunk_attn", lib().spc_kv4_chunk_attn(
        q, _dev("cache", cache, _BYTES, num_blocks * n_kv * block_size * SPC_KV4_RECORD, dev),
        _dev("block_table", block_table, _I32, B * max_blocks, dev), _dev("len", len, _I32, B, dev),
        _dev("cu_seqlens", cu_seqlens, _I32, B + 1, dev), T, B, n_q, n_kv, d, num_blocks, block_size, max_blocks, q_stride,
        float(scale), _dev("out", out, _BF16, T * n_q * d, dev), _dev("lse", lse, _F32, T * n_q, dev),
        _dev("workspace", workspace, _BYTES, workspace_bytes, dev), workspace_bytes, _raw_stream(stream, dev)))


def spc_kv4_attn_mass_workspace_size(T, B, n_q, n_kv, d) -> int:
    return int(lib().spc_kv4_attn_mass_workspace_size(T, B, n_q, n_kv, d))


def spc_kv4_attn_mass(q, cache, block_table, len, cu_seqlens, lse, mass_prev, mass_next, T, B, n_q, n_kv, d, num_blocks,
                      block_size, max_blocks, cap, scale, keep, workspace, workspace_bytes=None, q_stride=None,
                      stream=None) -> None:
    """The attention weight that the cached positions receive from new tokens
    (spc_kv4_chunk_attn's rows and lse), added to keep * mass_prev."""
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    dev = _device()
    q, q_stride = _rows("q", q, T, n_q, d, q_stride, dev)
    _check("spc_kv4_attn_mass", lib().spc_kv4_attn_mass(
        q, _dev("cache", cache, _BYTES, num_blocks * n_kv * block_size * SPC_KV4_RECORD, dev),
        _dev("block_table", block_table, _I32, B * max_blocks, dev), _dev("len", len, _I32, B, dev),
        _dev("cu_seqlens", cu_seqlens, _I32, B + 1, dev), _dev("lse", lse, _F32, T * n_q, dev),
        _dev("mass_prev", mass_prev, _F32, B * n_kv * cap, dev), _dev("mass_next", mass_next, _F32, B * n_kv * cap, dev),
        T, B, n_q, n_kv, d, num_blocks, block_size, max_blocks, cap, q_stride, float(scale), float(keep),
        _dev("workspace", workspace, _BYTES, workspace_bytes, dev), workspace_bytes, _raw_stream(stream, dev)))


def spc_kv4_evict(cache, block_table, block_table_next, len, len_next, mass, mass_next, kept, status, B, n_kv, d,
                  num_blocks, block_size, max_blocks, cap, budget, n_sink, n_recent, stream=None) -> None:
    """Eviction by accumulated attention weight: each KV head's kept records to
    the front of block_table_next's blocks (block_table's own to shrink in place)."""
    dev = _device()
    _check("spc_kv4_evict", lib().spc_kv4_evict(
        _dev("cache", cache, _BYTES, num_blocks * n_kv * block_size * SPC_KV4_RECORD, dev),
        _dev("block_table", block_table, _I32, B * max_blocks, dev),
        _dev("block_table_next", block_table_next, _I32, B * max_blocks, dev), _dev("len", len, _I32, B, dev),
        _dev("len_next", len_next, _I32, B, dev), _dev("mass", mass, _F32, B * n_kv * cap, dev),
        _dev("mass_next", mass_next, _F32, B * n_kv * cap, dev), _dev("kept", kept, _I32, B * n_kv * budget, dev),
        _dev("status", status, _I32, 1, dev), B, n_kv, d, num_blocks, block_size, max_blocks, cap, budget, n_sink, n_recent,
        _raw_stream(stream, dev)))


def spc_device_sm_count() -> int:
    return int(lib().spc_device_sm_count())


# ------------------------------------------------------------------ view tables
def gather_views(host_ptrs: Sequence[int], slot_ptrs: Sequence[int], layer0: Sequence[int],
                 n_layers: Sequence[int], store_layer0: Optional[Sequence[int]] = None,
                 store_layers: Optional[Sequence[int]] = None) -> np.ndarray:
    """spc_gather_view table. By default a request's store holds exactly its
    host layers (store_layer0 = layer0, store_layers = n_layers)."""
    v = np.zeros(len(host_ptrs), GATHER_VIEW_DTYPE)
    v["host"], v["slots"], v["layer0"], v["n_layers"] = host_ptrs, slot_ptrs, layer0, n_layers
    v["store_layer0"] = layer0 if store_layer0 is None else store_layer0
    v["store_layers"] = n_layers if store_layers is None else store_layers
    return v


def kv_views(k_ptrs, v_ptrs, rows, use_slots) -> np.ndarray:
    v = np.zeros(len(k_ptrs), KV_VIEW_DTYPE)
    v["k"], v["v"], v["rows"], v["use_slots"] = k_ptrs, v_ptrs, rows, use_slots
    return v


def to_device_bytes(arr: np.ndarray, device):
    import torch
    return torch.from_numpy(np.ascontiguousarray(arr).view(np.uint8).copy()).to(device)


__all__ = [n for n in dir() if n.startswith("spc_")] + [
    "SpcError", "lib", "gather_views", "kv_views", "to_device_bytes", "GATHER_VIEW_DTYPE",
    "KV_VIEW_DTYPE", "LIB_PATH", "SIGNATURES"]
