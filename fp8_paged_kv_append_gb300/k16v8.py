"""Thin Python binding of libk16v8.so (the C ABI in include/k16v8.h).

Argument marshalling only: shapes and strides are read from torch tensors,
device pointers and the current CUDA stream are passed through ctypes, and
every status is turned into an exception.  All computation runs in the
library's CUDA kernels; there is no fallback of any kind -- importing this
module on a machine without the built library raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libk16v8.so")

K16V8_OK = 0
K16V8_ERR_INVALID_ARG = 1
K16V8_ERR_UNSUPPORTED_SHAPE = 2
K16V8_ERR_WORKSPACE_TOO_SMALL = 3
K16V8_ERR_CUDA = 4
K16V8_ERR_DEVICE_BOUNDS = 5
K16V8_ERR_STATIC_SCRATCH_LIMIT = 6
STATIC_SCRATCH_BYTES = 32 << 20
K16V8_F16 = 0
K16V8_F32 = 1
K16V8_BF16 = 2
DECODE_METADATA_READY = 1
DEVERR_SLOT, DEVERR_PAGE, DEVERR_SEQLEN, DEVERR_TIMEOUT, DEVERR_INTERNAL = 1, 2, 4, 8, 16
DEVERR_POSITION, DEVERR_TREE, DEVERR_PROBS = 32, 64, 128
PAGE_SIZE = 16
HEAD_DIM = 128
MAX_SPLIT_CHUNK = 8192  # K16V8_MAX_SPLIT_CHUNK
MAX_TREE_NODES = 64  # K16V8_MAX_TREE_NODES
MAX_ROPE_AXES = 4  # K16V8_MAX_ROPE_AXES

# Every symbol include/k16v8.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_i32, _i64, _sz, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "k16v8_kv_append": (_i32, [_P, _i64, _P, _i32, _i64, _P, _i32, _P, _P, _P, _i32, _i32,
                               _i32, _P, _P]),
    "k16v8_decode_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
    "k16v8_decode_workspace_layout": (_i32, [_i32, _i32, _i32, _i32, _i32,
                                             ctypes.POINTER(_sz), ctypes.POINTER(_sz),
                                             ctypes.POINTER(_i32)]),
    "k16v8_paged_decode_split": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32, _i32, _i32,
                                        _i32, _i32, _f32, _i32, _P, _sz, _P, _P]),
    "k16v8_merge_states": (_i32, [_P, _P, _i32, _i32, _i32, _i32, _P, _i32, _P, _P, _P]),
    "k16v8_paged_decode_attention": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32, _i32,
                                            _i32, _i32, _i32, _f32, _i32, _P, _sz, _P, _P,
                                            _P, _P]),
    "k16v8_paged_decode_attention_static": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32,
                                                   _i32, _i32, _i32, _i32, _f32, _i32, _P, _P,
                                                   _P, _P]),
    "k16v8_paged_decode_append_split": (_i32, [_P, _P, _P, _P, _P, _P, _P, _i32, _P, _i32, _i32,
                                               _i32, _i32, _i32, _i32, _f32, _i32, _P, _sz, _P,
                                               _P]),
    "k16v8_paged_decode_append_attention": (_i32, [_P, _P, _P, _P, _P, _P, _P, _i32, _P, _i32,
                                                   _i32, _i32, _i32, _i32, _i32, _f32, _i32, _P,
                                                   _sz, _P, _P, _P, _P]),
    "k16v8_kv_append_v16": (_i32, [_P, _i64, _P, _i64, _P, _i32, _P, _P, _i32, _i32, _i32, _P,
                                   _P]),
    "k16v8_paged_decode_split_v16": (_i32, [_P, _P, _P, _P, _i32, _P, _i32, _i32, _i32, _i32,
                                            _i32, _i32, _f32, _i32, _P, _sz, _P, _P]),
    "k16v8_paged_decode_attention_v16": (_i32, [_P, _P, _P, _P, _i32, _P, _i32, _i32, _i32,
                                                _i32, _i32, _i32, _f32, _i32, _P, _sz, _P, _P,
                                                _P, _P]),
    "k16v8_paged_prefill_attention": (_i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _i32, _P,
                                             _i32, _i32, _i32, _i32, _i32, _f32, _P, _P, _P,
                                             _P]),
    "k16v8_prefill_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "k16v8_paged_prefill_attention_split": (_i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _i32,
                                                   _P, _i32, _i32, _i32, _i32, _i32, _f32,
                                                   _i32, _i32, _P, _sz, _P, _P, _P, _P]),
    "k16v8_decode_balanced_workspace_size": (_sz, [_i32, _i32, _i32]),
    "k16v8_paged_decode_attention_balanced": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32,
                                                     _i32, _i32, _i32, _f32, _P, _sz, _P, _P,
                                                     _i32, _P, _P]),
    "k16v8_paged_decode_balanced_split": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32,
                                                 _i32, _i32, _i32, _f32, _P, _sz, _P, _P, _i32,
                                                 _P, _P]),
    "k16v8_merge_balanced": (_i32, [_P, _sz, _i32, _i32, _i32, _i32, _P, _P, _P]),
    "k16v8_paged_decode_append_balanced_split": (_i32, [_P, _P, _P, _P, _P, _P, _P, _i32, _P,
                                                        _i32, _i32, _i32, _i32, _i32, _f32, _P,
                                                        _sz, _P, _P, _i32, _P, _P]),
    "k16v8_paged_decode_append_attention_balanced": (_i32, [_P, _P, _P, _P, _P, _P, _P, _i32,
                                                            _P, _i32, _i32, _i32, _i32, _i32,
                                                            _f32, _P, _sz, _P, _P, _i32, _P,
                                                            _P]),
    "k16v8_paged_decode_split_wait_test": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32,
                                                  _i32, _i32, _i32, _i32, _f32, _i32, _P, _sz,
                                                  _P, _P]),
    "k16v8_paged_prefill_attention_wait_test": (_i32, [_P, _P, _i32, _i32, _P, _P, _P, _P,
                                                       _i32, _P, _i32, _i32, _i32, _i32, _i32,
                                                       _f32, _P, _P, _P, _P]),
    "k16v8_rope_kv_append": (_i32, [_P, _i64, _P, _i64, _P, _i64, _i32, _P, _P, _i32, _i32, _f32,
                                    _P, _i32, _P, _P, _P, _P, _i32, _i32, _i32, _i32, _P, _P]),
    "k16v8_rope_axes_kv_append": (_i32, [_P, _i64, _P, _i64, _P, _i64, _i32, _P, _i32, _P, _P, _i32,
                                         _i32, _f32, _P, _i32, _P, _P, _P, _P, _i32, _i32, _i32,
                                         _i32, _P, _P]),
    "k16v8_rope_kv_append_k8v8": (_i32, [_P, _i64, _P, _i64, _P, _i64, _i32, _P, _i32, _P, _i32, _P,
                                         _P, _i32, _i32, _f32, _P, _i32, _P, _i32, _P, _P, _P, _P,
                                         _i32, _i32, _i32, _i32, _P, _P]),
    "k16v8_decode_workspace_size_k8v8": (_sz, [_i32, _i32, _i32]),
    "k16v8_paged_decode_attention_k8v8": (_i32, [_P, _P, _P, _P, _P, _i32, _P, _i32, _i32, _i32, _i32,
                                                 _i32, _f32, _P, _sz, _P, _P, _P, _P]),
    "k16v8_attention_workspace_size_k8v8": (_sz, [_i32, _i32, _i32, _i32]),
    "k16v8_paged_prefill_attention_k8v8": (
        _i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _i32, _P,
               _i32, _i32, _i32, _i32, _i32, _i32, _f32, _P, _sz, _P, _P,
               _P, _P]),
    "k16v8_paged_cross_attention_k8v8": (
        _i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _i32, _P,
               _i32, _i32, _i32, _i32, _i32, _i32, _f32, _P, _sz, _P, _P,
               _P, _P]),
    "k16v8_paged_prefill_attention_k8v8_wait_test": (
        _i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _i32, _P,
               _i32, _i32, _i32, _i32, _i32, _i32, _f32, _P, _sz, _P, _P,
               _P, _P]),
    "k16v8_tree_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "k16v8_paged_tree_attention": (_i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _P, _i32, _P, _i32,
                                          _i32, _i32, _i32, _i32, _i32, _f32, _P, _sz, _P, _P, _P,
                                          _P]),
    "k16v8_paged_tree_attention_wait_test": (_i32, [_P, _P, _i32, _i32, _P, _P, _P, _P, _P, _i32, _P,
                                                    _i32, _i32, _i32, _i32, _i32, _i32, _f32, _P,
                                                    _sz, _P, _P, _P, _P]),
    "k16v8_tree_verify": (_i32, [_P, _i64, _P, _i64, _P, _P, _P, _i32, _i32, _P, _i32, _i32, _P,
                                 _P, _P, _P, _P]),
    "k16v8_kv_compact": (_i32, [_P, _P, _i32, _P, _i32, _P, _P, _P, _i32, _P, _i32, _i32, _i32,
                                _i32, _P, _P, _P]),
    "k16v8_read_device_error": (_i32, [_P, _P, ctypes.POINTER(_i32)]),
    "k16v8_status_string": (ctypes.c_char_p, [_i32]),
}

_lib = None


class K16V8Error(RuntimeError):
    def __init__(self, name: str, status: int):
        self.status = status
        super().__init__(f"{name}: {status_string(status)} (status {status})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libk16v8.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(
                f"libk16v8.so not found at {path}: build it with "
                "`python -m fp8_paged_kv_append_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load_library().k16v8_status_string(int(status)).decode()


k16v8_status_string = status_string


def _check(name: str, status: int) -> None:
    if status != K16V8_OK:
        raise K16V8Error(name, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return _stream_on(None, torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_on(stream, dev: int) -> int:
    """The handle of a stream, None being the current one of device dev (the
    handle alone: building the Stream object costs 3 us)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _row_stride(t: torch.Tensor, name: str) -> int:
    if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with dense rows")
    return t.stride(0)


_F16, _F32, _U8, _I32, _I64 = (torch.float16, torch.float32, torch.uint8, torch.int32,
                                torch.int64)


def _device(t: torch.Tensor) -> int:
    """The current device, on which the tensors of a call have to be."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current CUDA device, got {t.device}")
    return dev


def _dense(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a dense tensor of this type and shape on device dev."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name} must be a dense {dtype} tensor of shape {tuple(shape)} on "
                     f"cuda:{dev}, got {t.dtype} {tuple(t.shape)}"
                     f"{'' if t.is_contiguous() else ' (strided)'} on {t.device}")


def _rows(t, name: str, dtype, shape, dev: int) -> int:
    """Token stride of [tokens, heads, head_dim] with dense rows (a slice of a
    wider row is fine), 0 for a single token."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        ts, hs, ds = t.stride()
        if ds == 1 and (hs == shape[2] or shape[1] == 1):
            if shape[0] <= 1:
                return 0
            if ts >= shape[1] * shape[2]:
                return ts
    raise ValueError(f"{name} must be {dtype} {tuple(shape)} with dense rows on cuda:{dev}, got "
                     f"{t.dtype} {tuple(t.shape)}, strides {t.stride()} on {t.device}")


def _error_word(dev_error, dev: int):
    return None if dev_error is None else _dense(dev_error, "dev_error", _I32, (1,), dev)


# ---- kv_append ---------------------------------------------------------------

def k16v8_kv_append(k, v, slot_mapping, v_scale, k_cache, v_cache, dev_error=None,
                    stream=None) -> None:
    """k fp16 [T,Hkv,D]; v fp16/fp32 [T,Hkv,D] (token stride may exceed the
    row, e.g. a slice of a fused QKV); slot_mapping int64 [T]; v_scale fp32
    [Hkv]; k_cache fp16 / v_cache uint8 [P,Hkv,16,D]."""
    T, hkv, d = k.shape
    vd = {torch.float16: K16V8_F16, torch.float32: K16V8_F32}[v.dtype]
    st = load_library().k16v8_kv_append(
        _ptr(k), _row_stride(k, "k"), _ptr(v), vd, _row_stride(v, "v"), _ptr(slot_mapping), T,
        _ptr(v_scale), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], hkv, d,
        _ptr(dev_error), _stream(stream))
    _check("k16v8_kv_append", st)


# ---- decode --------------------------------------------------------------------

def k16v8_decode_workspace_size(batch, num_qo_heads, head_dim, max_seq_len, split_chunk) -> int:
    return int(load_library().k16v8_decode_workspace_size(batch, num_qo_heads, head_dim,
                                                          max_seq_len, split_chunk))


def k16v8_decode_workspace_layout(batch, num_qo_heads, head_dim, max_seq_len, split_chunk):
    """(partial_o byte offset, partial_lse byte offset, max_chunks)."""
    o, l, c = _sz(), _sz(), _i32()
    st = load_library().k16v8_decode_workspace_layout(
        batch, num_qo_heads, head_dim, max_seq_len, split_chunk,
        ctypes.byref(o), ctypes.byref(l), ctypes.byref(c))
    _check("k16v8_decode_workspace_layout", st)
    return o.value, l.value, c.value


def workspace_views(workspace, batch, num_qo_heads, head_dim, max_seq_len, split_chunk):
    """fp32 views (partial_o [B,Hq,C,D], partial_lse [B,Hq,C]) of a workspace."""
    o_off, l_off, C = k16v8_decode_workspace_layout(batch, num_qo_heads, head_dim,
                                                    max_seq_len, split_chunk)
    n = batch * num_qo_heads * C
    po = workspace[o_off:o_off + n * head_dim * 4].view(torch.float32)
    pl = workspace[l_off:l_off + n * 4].view(torch.float32)
    return po.view(batch, num_qo_heads, C, head_dim), pl.view(batch, num_qo_heads, C)


def k16v8_paged_decode_split(q, k_cache, v_cache, v_scale, block_table, seq_lens, max_seq_len,
                             sm_scale, split_chunk, workspace, dev_error=None, stream=None):
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_split(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, hq, k_cache.shape[1], d,
        k_cache.shape[0], float(sm_scale), int(split_chunk), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_split", st)


def k16v8_paged_decode_split_wait_test(q, k_cache, v_cache, v_scale, block_table, seq_lens,
                                       max_seq_len, sm_scale, split_chunk, workspace,
                                       dev_error=None, stream=None):
    """Test hook: k16v8_paged_decode_split with one page copy of the first CTA
    withheld, so that CTA's bounded wait expires (K16V8_DEVERR_TIMEOUT)."""
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_split_wait_test(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, hq, k_cache.shape[1], d,
        k_cache.shape[0], float(sm_scale), int(split_chunk), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_split_wait_test", st)


def k16v8_merge_states(partial_o, partial_lse, seq_lens, split_chunk, out, lse=None,
                       stream=None):
    B, hq, C, d = partial_o.shape
    st = load_library().k16v8_merge_states(
        _ptr(partial_o), _ptr(partial_lse), B, hq, C, d, _ptr(seq_lens), int(split_chunk),
        _ptr(out), _ptr(lse), _stream(stream))
    _check("k16v8_merge_states", st)


def k16v8_paged_decode_attention(q, k_cache, v_cache, v_scale, block_table, seq_lens,
                                 max_seq_len, sm_scale, split_chunk, workspace, out, lse=None,
                                 dev_error=None, stream=None):
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_attention(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, hq, k_cache.shape[1], d,
        k_cache.shape[0], float(sm_scale), int(split_chunk), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _ptr(dev_error),
        _stream(stream))
    _check("k16v8_paged_decode_attention", st)


def k16v8_paged_decode_append_split(q, k_new, v_new, k_cache, v_cache, v_scale, block_table,
                                    seq_lens, max_seq_len, sm_scale, split_chunk, workspace,
                                    dev_error=None, stream=None):
    """Decode split with each sequence's new token (k_new / v_new fp16
    [B, Hkv, D]) written at position seq_lens[b] - 1 by the same kernel."""
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_append_split(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale),
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, hq,
        k_cache.shape[1], d, k_cache.shape[0], float(sm_scale), int(split_chunk),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_error),
        _stream(stream))
    _check("k16v8_paged_decode_append_split", st)


def k16v8_paged_decode_append_attention(q, k_new, v_new, k_cache, v_cache, v_scale, block_table,
                                        seq_lens, max_seq_len, sm_scale, split_chunk, workspace,
                                        out, lse=None, dev_error=None, stream=None):
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_append_attention(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale),
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, hq,
        k_cache.shape[1], d, k_cache.shape[0], float(sm_scale), int(split_chunk),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
        _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_append_attention", st)


def k16v8_kv_append_v16(k, v, slot_mapping, k_cache, v_cache16, dev_error=None, stream=None):
    """FP16-KV control cache write (values copied as fp16)."""
    T, hkv, d = k.shape
    st = load_library().k16v8_kv_append_v16(
        _ptr(k), _row_stride(k, "k"), _ptr(v), _row_stride(v, "v"), _ptr(slot_mapping), T,
        _ptr(k_cache), _ptr(v_cache16), k_cache.shape[0], hkv, d, _ptr(dev_error),
        _stream(stream))
    _check("k16v8_kv_append_v16", st)


def k16v8_paged_decode_split_v16(q, k_cache, v_cache16, block_table, seq_lens, max_seq_len,
                                 sm_scale, split_chunk, workspace, dev_error=None, stream=None):
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_split_v16(
        _ptr(q), _ptr(k_cache), _ptr(v_cache16), _ptr(block_table), block_table.shape[1],
        _ptr(seq_lens), int(max_seq_len), B, hq, k_cache.shape[1], d, k_cache.shape[0],
        float(sm_scale), int(split_chunk), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_split_v16", st)


def k16v8_paged_decode_attention_v16(q, k_cache, v_cache16, block_table, seq_lens, max_seq_len,
                                     sm_scale, split_chunk, workspace, out, lse=None,
                                     dev_error=None, stream=None):
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_attention_v16(
        _ptr(q), _ptr(k_cache), _ptr(v_cache16), _ptr(block_table), block_table.shape[1],
        _ptr(seq_lens), int(max_seq_len), B, hq, k_cache.shape[1], d, k_cache.shape[0],
        float(sm_scale), int(split_chunk), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), _ptr(dev_error),
        _stream(stream))
    _check("k16v8_paged_decode_attention_v16", st)


def k16v8_paged_prefill_attention(q, qo_indptr, max_qlen, k_cache, v_cache, v_scale,
                                  block_table, seq_lens, sm_scale, out, lse=None, dev_error=None,
                                  stream=None):
    """Causal attention of q [total_q, Hq, D] (ragged by qo_indptr [B+1])
    against the paged cache, whose seq_lens include these new tokens."""
    total_q, hq, d = q.shape
    st = load_library().k16v8_paged_prefill_attention(
        _ptr(q), _ptr(qo_indptr), total_q, int(max_qlen), _ptr(k_cache), _ptr(v_cache),
        _ptr(v_scale), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        seq_lens.shape[0], hq, k_cache.shape[1], d, k_cache.shape[0], float(sm_scale), _ptr(out),
        _ptr(lse), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_prefill_attention", st)


def k16v8_paged_prefill_attention_wait_test(q, qo_indptr, max_qlen, k_cache, v_cache, v_scale,
                                            block_table, seq_lens, sm_scale, out, lse=None,
                                            dev_error=None, stream=None):
    """Test hook: k16v8_paged_prefill_attention with the first KV tile of the
    first CTA withheld, so that CTA's bounded wait expires
    (K16V8_DEVERR_TIMEOUT)."""
    total_q, hq, d = q.shape
    st = load_library().k16v8_paged_prefill_attention_wait_test(
        _ptr(q), _ptr(qo_indptr), total_q, int(max_qlen), _ptr(k_cache), _ptr(v_cache),
        _ptr(v_scale), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        seq_lens.shape[0], hq, k_cache.shape[1], d, k_cache.shape[0], float(sm_scale), _ptr(out),
        _ptr(lse), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_prefill_attention_wait_test", st)


def k16v8_prefill_workspace_size(max_qlen, batch, num_qo_heads, num_kv_heads, head_dim,
                                 kv_splits=0, max_seq_len=0) -> int:
    """Bytes of workspace k16v8_paged_prefill_attention_split needs (0: the
    call will not split, no workspace needed)."""
    return int(load_library().k16v8_prefill_workspace_size(max_qlen, batch, num_qo_heads,
                                                            num_kv_heads, head_dim, kv_splits,
                                                            max_seq_len))


def k16v8_paged_prefill_attention_split(q, qo_indptr, max_qlen, k_cache, v_cache, v_scale,
                                        block_table, seq_lens, sm_scale, workspace, out,
                                        lse=None, dev_error=None, stream=None, kv_splits=0,
                                        max_seq_len=0):
    """Prefill attention with the KV range of each query-tile pair cut into
    up to 4 parts (merged in the kernel) when the call has too few pairs to
    fill the GPU; `workspace` zero-filled before its first use."""
    total_q, hq, d = q.shape
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().k16v8_paged_prefill_attention_split(
        _ptr(q), _ptr(qo_indptr), total_q, int(max_qlen), _ptr(k_cache), _ptr(v_cache),
        _ptr(v_scale), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        seq_lens.shape[0], hq, k_cache.shape[1], d, k_cache.shape[0], float(sm_scale),
        int(kv_splits), int(max_seq_len), _ptr(workspace), nbytes, _ptr(out), _ptr(lse),
        _ptr(dev_error),
        _stream(stream))
    _check("k16v8_paged_prefill_attention_split", st)


def k16v8_paged_decode_attention_static(q, k_cache, v_cache, v_scale, block_table, seq_lens,
                                        max_seq_len, sm_scale, split_chunk, out, lse=None,
                                        dev_error=None, stream=None):
    """Decode attention with the partials in the library's built-in device
    scratch: for callers that cannot allocate device memory.  Calls that
    overlap on the GPU race on that scratch; the first call on a device
    should come before any stream capture."""
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_attention_static(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), int(max_seq_len), B, hq, k_cache.shape[1], d,
        k_cache.shape[0], float(sm_scale), int(split_chunk), _ptr(out), _ptr(lse),
        _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_attention_static", st)


def k16v8_decode_balanced_workspace_size(batch, num_qo_heads, head_dim) -> int:
    """Bytes of workspace k16v8_paged_decode_attention_balanced needs on the
    current device (0 for an unsupported shape)."""
    return int(load_library().k16v8_decode_balanced_workspace_size(batch, num_qo_heads, head_dim))


def k16v8_paged_decode_attention_balanced(q, k_cache, v_cache, v_scale, block_table, seq_lens,
                                          sm_scale, workspace, out, lse=None, dev_error=None,
                                          stream=None, flags=0):
    """Decode attention with every CTA given the same number of KV tiles."""
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_attention_balanced(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), B, hq, k_cache.shape[1], d, k_cache.shape[0],
        float(sm_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(out), _ptr(lse), int(flags), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_attention_balanced", st)


def k16v8_paged_decode_balanced_split(q, k_cache, v_cache, v_scale, block_table, seq_lens,
                                      sm_scale, workspace, out, lse=None, dev_error=None,
                                      stream=None, flags=0):
    B, hq, d = q.shape
    st = load_library().k16v8_paged_decode_balanced_split(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale), _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), B, hq, k_cache.shape[1], d, k_cache.shape[0],
        float(sm_scale), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(out), _ptr(lse), int(flags), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_decode_balanced_split", st)


def k16v8_merge_balanced(workspace, num_kv_heads, out, lse=None, stream=None):
    B, hq, d = out.shape
    st = load_library().k16v8_merge_balanced(
        _ptr(workspace), workspace.numel() * workspace.element_size(), B, hq, int(num_kv_heads),
        d, _ptr(out), _ptr(lse), _stream(stream))
    _check("k16v8_merge_balanced", st)


def _append_balanced(name, q, k_new, v_new, k_cache, v_cache, v_scale, block_table, seq_lens,
                     sm_scale, workspace, out, lse, dev_error, stream, flags):
    B, hq, d = q.shape
    st = getattr(load_library(), name)(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(v_scale),
        _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, hq, k_cache.shape[1], d,
        k_cache.shape[0], float(sm_scale), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse), int(flags),
        _ptr(dev_error), _stream(stream))
    _check(name, st)


def k16v8_paged_decode_append_balanced_split(q, k_new, v_new, k_cache, v_cache, v_scale,
                                             block_table, seq_lens, sm_scale, workspace, out,
                                             lse=None, dev_error=None, stream=None, flags=0):
    """Load-balanced decode split with each sequence's new token (k_new,
    v_new [B, Hkv, D] fp16) written into the cache by the same kernel."""
    _append_balanced("k16v8_paged_decode_append_balanced_split", q, k_new, v_new, k_cache,
                     v_cache, v_scale, block_table, seq_lens, sm_scale, workspace, out, lse,
                     dev_error, stream, flags)


def k16v8_paged_decode_append_attention_balanced(q, k_new, v_new, k_cache, v_cache, v_scale,
                                                 block_table, seq_lens, sm_scale, workspace, out,
                                                 lse=None, dev_error=None, stream=None, flags=0):
    """k16v8_paged_decode_append_balanced_split followed by the merge."""
    _append_balanced("k16v8_paged_decode_append_attention_balanced", q, k_new, v_new, k_cache,
                     v_cache, v_scale, block_table, seq_lens, sm_scale, workspace, out, lse,
                     dev_error, stream, flags)


# ---- speculative step ------------------------------------------------------------

_X_DTYPES = {torch.float16: K16V8_F16, torch.float32: K16V8_F32, torch.bfloat16: K16V8_BF16}


def k16v8_rope_kv_append(q, k, v, positions, inv_freq, slot_mapping, v_scale, q_out, k_cache,
                         v_cache, interleaved=False, attn_factor=1.0, dev_error=None,
                         stream=None) -> None:
    """Rotary positions fused with the cache write: q [T,Hq,D] (or None), k, v
    [T,Hkv,D] of one type (fp16, fp32 or bf16; token strides may exceed the
    row, e.g. slices of a fused QKV); positions int32 [T]; inv_freq fp32
    [rotary_dim/2] (see rope.rope_inv_freq); slot_mapping int64 [T]; q_out
    fp16 [T,Hq,D] (q itself if that is dense fp16); caches as for
    k16v8_kv_append."""
    T, hkv, d = k.shape
    dt, dev = k.dtype, _device(k)
    if dt not in _X_DTYPES:
        raise ValueError(f"k must be fp16, fp32 or bf16, got {dt}")
    hq = 0 if q is None else q.shape[1]
    if q is None:
        q_ptr, q_ts, out_ptr = None, 0, None
    else:
        q_ptr, q_ts = q.data_ptr(), _rows(q, "q", dt, (T, hq, d), dev)
        out_ptr = _dense(q_out, "q_out", _F16, (T, hq, d), dev)
    row, tokens = (T, hkv, d), (T,)
    cache = (k_cache.shape[0], hkv, PAGE_SIZE, d)
    half = inv_freq.numel()
    st = (_lib or load_library()).k16v8_rope_kv_append(
        q_ptr, q_ts, k.data_ptr(), _rows(k, "k", dt, row, dev), v.data_ptr(),
        _rows(v, "v", dt, row, dev), _X_DTYPES[dt],
        _dense(positions, "positions", _I32, tokens, dev),
        _dense(inv_freq, "inv_freq", _F32, (half,), dev), 2 * half, 1 if interleaved else 0,
        attn_factor, _dense(slot_mapping, "slot_mapping", _I64, tokens, dev), T,
        _dense(v_scale, "v_scale", _F32, (hkv,), dev),
        out_ptr,
        _dense(k_cache, "k_cache", _F16, cache, dev),
        _dense(v_cache, "v_cache", _U8, cache, dev), cache[0], hq, hkv, d,
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_rope_kv_append", st)


def k16v8_tree_workspace_size(total_q, batch, max_nodes, num_qo_heads, num_kv_heads, head_dim,
                              max_seq_len) -> int:
    """Bytes of workspace k16v8_paged_tree_attention needs for these sizes on
    the current device (0 where they are refused)."""
    return int(load_library().k16v8_tree_workspace_size(
        total_q, batch, max_nodes, num_qo_heads, num_kv_heads, head_dim, max_seq_len))


def k16v8_paged_tree_attention(q, qo_indptr, max_nodes, tree_mask, k_cache, v_cache, v_scale,
                               block_table, seq_lens, max_seq_len, sm_scale, workspace, out,
                               lse=None, dev_error=None, stream=None) -> None:
    """Attention of drafted trees: q fp16 [total_q,Hq,D], ragged by qo_indptr
    int32 [B+1], the nodes being the last positions of the cache; tree_mask
    int64 [total_q], bit j of a node's word set where it sees node j of its
    tree (tree_step.tree_masks builds it from the parents).  workspace uint8
    of k16v8_tree_workspace_size bytes, not shared by calls that overlap."""
    total_q, hq, d = q.shape
    dev = _device(q)
    P, hkv = k_cache.shape[0], k_cache.shape[1]
    B = seq_lens.shape[0]
    cache = (P, hkv, PAGE_SIZE, d)
    maxp = block_table.shape[1]
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws = _dense(workspace, "workspace", workspace.dtype, workspace.shape, dev)
    st = (_lib or load_library()).k16v8_paged_tree_attention(
        _dense(q, "q", _F16, (total_q, hq, d), dev),
        _dense(qo_indptr, "qo_indptr", _I32, (B + 1,), dev), total_q, max_nodes,
        _dense(tree_mask, "tree_mask", _I64, (total_q,), dev),
        _dense(k_cache, "k_cache", _F16, cache, dev),
        _dense(v_cache, "v_cache", _U8, cache, dev),
        _dense(v_scale, "v_scale", _F32, (hkv,), dev),
        _dense(block_table, "block_table", _I32, (B, maxp), dev), maxp,
        _dense(seq_lens, "seq_lens", _I32, (B,), dev), max_seq_len, B, hq, hkv, d, P,
        sm_scale, ws, ws_bytes, _dense(out, "out", _F16, (total_q, hq, d), dev),
        None if lse is None else _dense(lse, "lse", _F32, (total_q, hq), dev),
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_paged_tree_attention", st)


def k16v8_paged_tree_attention_wait_test(q, qo_indptr, max_nodes, tree_mask, k_cache, v_cache,
                                         v_scale, block_table, seq_lens, max_seq_len, sm_scale,
                                         workspace, out, lse=None, dev_error=None, stream=None):
    """Test hook: k16v8_paged_tree_attention with the keys of the first CTA's
    first tile withheld, so that CTA's bounded wait expires
    (K16V8_DEVERR_TIMEOUT)."""
    total_q, hq, d = q.shape
    st = load_library().k16v8_paged_tree_attention_wait_test(
        _ptr(q), _ptr(qo_indptr), total_q, int(max_nodes), _ptr(tree_mask), _ptr(k_cache),
        _ptr(v_cache), _ptr(v_scale), _ptr(block_table), block_table.shape[1], _ptr(seq_lens),
        int(max_seq_len), seq_lens.shape[0], hq, k_cache.shape[1], d, k_cache.shape[0],
        float(sm_scale), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
        _ptr(lse), _ptr(dev_error), _stream(stream))
    _check("k16v8_paged_tree_attention_wait_test", st)


def _prob_rows(t, name: str, shape, dev: int) -> int:
    """Row stride of fp32 [total_q, V] with dense rows, 0 for a single row."""
    if t.dtype is _F32 and t.shape == shape and t.get_device() == dev:
        rs, cs = t.stride()
        if cs == 1 or shape[1] == 1:
            if shape[0] <= 1:
                return 0
            if rs >= shape[1]:
                return rs
    raise ValueError(f"{name} must be float32 {tuple(shape)} with dense rows on cuda:{dev}, got "
                     f"{t.dtype} {tuple(t.shape)}, strides {t.stride()} on {t.device}")


def k16v8_tree_verify(target_probs, draft_probs, tokens, parents, qo_indptr, max_nodes, uniforms,
                      path, path_len, next_token, dev_error=None, stream=None) -> None:
    """Accepted path and next token of every tree: target_probs, draft_probs
    fp32 [total_q,V] (rows may be strided; draft_probs None where the drafts
    were not sampled); tokens, parents int32 [total_q]; uniforms fp32
    [total_q] in [0, 1); writes path int32 [B,max_nodes], path_len int32 [B],
    next_token int32 [B]."""
    total_q, V = target_probs.shape
    dev = _device(target_probs)
    B = path_len.shape[0]
    shape, rows, seqs = (total_q, V), (total_q,), (B,)
    st = (_lib or load_library()).k16v8_tree_verify(
        target_probs.data_ptr(), _prob_rows(target_probs, "target_probs", shape, dev),
        None if draft_probs is None else draft_probs.data_ptr(),
        0 if draft_probs is None else _prob_rows(draft_probs, "draft_probs", shape, dev),
        _dense(tokens, "tokens", _I32, rows, dev),
        _dense(parents, "parents", _I32, rows, dev),
        _dense(qo_indptr, "qo_indptr", _I32, (B + 1,), dev), total_q, max_nodes,
        _dense(uniforms, "uniforms", _F32, rows, dev), V, B,
        _dense(path, "path", _I32, (B, max_nodes), dev),
        _dense(path_len, "path_len", _I32, seqs, dev),
        _dense(next_token, "next_token", _I32, seqs, dev), _error_word(dev_error, dev),
        _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_tree_verify", st)


def layer_pointers(caches) -> torch.Tensor:
    """Device array of the layers' cache addresses for k16v8_kv_compact (the
    caches must outlive it)."""
    return torch.tensor([c.data_ptr() for c in caches], dtype=torch.int64,
                        device=caches[0].device)


def k16v8_kv_compact(k_ptrs, v_ptrs, num_pages, num_kv_heads, head_dim, block_table, seq_lens,
                     qo_indptr, path, path_len, new_seq_lens=None, dev_error=None,
                     stream=None) -> None:
    """Move the accepted rows of every tree to the front of its positions in
    all layers (k_ptrs, v_ptrs: layer_pointers of the caches, each of
    num_pages pages); path int32 [B,max_nodes], path_len int32 [B] from
    k16v8_tree_verify; new_seq_lens int32 [B] (none of the inputs)."""
    dev = _device(k_ptrs)
    layers = k_ptrs.shape[0]
    B, max_nodes = path.shape
    maxp = block_table.shape[1]
    st = (_lib or load_library()).k16v8_kv_compact(
        _dense(k_ptrs, "k_ptrs", _I64, (layers,), dev),
        _dense(v_ptrs, "v_ptrs", _I64, (layers,), dev), layers,
        _dense(block_table, "block_table", _I32, (B, maxp), dev), maxp,
        _dense(seq_lens, "seq_lens", _I32, (B,), dev),
        _dense(qo_indptr, "qo_indptr", _I32, (B + 1,), dev),
        _dense(path, "path", _I32, (B, max_nodes), dev), max_nodes,
        _dense(path_len, "path_len", _I32, (B,), dev), B, num_kv_heads, head_dim,
        num_pages,
        None if new_seq_lens is None else _dense(new_seq_lens, "new_seq_lens", _I32, (B,),
                                                 dev),
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_kv_compact", st)


# ---- positions with several axes; the K8/V8 cache ------------------------------------

def _axes(pair_axis, half: int) -> bytes:
    """The axis of each pair as the host array of the C ABI (bytes are taken as
    they are)."""
    if type(pair_axis) is not bytes:
        # (by its entries: bytes() of an array would be its memory, of a number zeros)
        pair_axis = bytes(list(pair_axis))
    if len(pair_axis) != half:
        raise ValueError(f"pair_axis must have an entry for each of {half} pairs, got "
                         f"{len(pair_axis)}")
    return pair_axis


def k16v8_rope_axes_kv_append(q, k, v, positions, pair_axis, inv_freq, slot_mapping, v_scale, q_out,
                              k_cache, v_cache, interleaved=False, attn_factor=1.0, dev_error=None,
                              stream=None) -> None:
    """k16v8_rope_kv_append with positions int32 [axes,T]: pair i is turned by
    row pair_axis[i] of them (host integers, e.g. rope.rope_pair_axes)."""
    T, hkv, d = k.shape
    dt, dev = k.dtype, _device(k)
    if dt not in _X_DTYPES:
        raise ValueError(f"k must be fp16, fp32 or bf16, got {dt}")
    hq = 0 if q is None else q.shape[1]
    if q is None:
        q_ptr, q_ts, out_ptr = None, 0, None
    else:
        q_ptr, q_ts = q.data_ptr(), _rows(q, "q", dt, (T, hq, d), dev)
        out_ptr = _dense(q_out, "q_out", _F16, (T, hq, d), dev)
    row = (T, hkv, d)
    cache = (k_cache.shape[0], hkv, PAGE_SIZE, d)
    half, axes = inv_freq.numel(), positions.shape[0]
    st = (_lib or load_library()).k16v8_rope_axes_kv_append(
        q_ptr, q_ts, k.data_ptr(), _rows(k, "k", dt, row, dev), v.data_ptr(),
        _rows(v, "v", dt, row, dev), _X_DTYPES[dt],
        _dense(positions, "positions", _I32, (axes, T), dev), axes, _axes(pair_axis, half),
        _dense(inv_freq, "inv_freq", _F32, (half,), dev), 2 * half, 1 if interleaved else 0,
        attn_factor, _dense(slot_mapping, "slot_mapping", _I64, (T,), dev), T,
        _dense(v_scale, "v_scale", _F32, (hkv,), dev), out_ptr,
        _dense(k_cache, "k_cache", _F16, cache, dev),
        _dense(v_cache, "v_cache", _U8, cache, dev), cache[0], hq, hkv, d,
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_rope_axes_kv_append", st)


def k16v8_rope_kv_append_k8v8(q, k, v, qo_indptr, positions, pair_axis, inv_freq, block_table,
                              seq_lens, q_out, k_cache, v_cache, kv_scale, interleaved=False,
                              attn_factor=1.0, dev_error=None, stream=None) -> None:
    """The K8/V8 cache write: q [T,Hq,D] (or None), k, v [T,Hkv,D] as for
    k16v8_rope_axes_kv_append, rows of sequence b being qo_indptr[b] ..
    qo_indptr[b+1] - 1 (int32 [B+1]) and its last positions of seq_lens int32
    [B]; positions int32 [axes,T], pair_axis and inv_freq as there, or None
    for rows that are not turned; k_cache, v_cache uint8 [P,Hkv,16,D],
    kv_scale fp32 [P,Hkv,2]."""
    T, hkv, d = k.shape
    dt, dev = k.dtype, _device(k)
    if dt not in _X_DTYPES:
        raise ValueError(f"k must be fp16, fp32 or bf16, got {dt}")
    hq = 0 if q is None else q.shape[1]
    if q is None:
        q_ptr, q_ts, out_ptr = None, 0, None
    else:
        q_ptr, q_ts = q.data_ptr(), _rows(q, "q", dt, (T, hq, d), dev)
        out_ptr = _dense(q_out, "q_out", _F16, (T, hq, d), dev)
    row, (B, maxp) = (T, hkv, d), block_table.shape
    P = k_cache.shape[0]
    cache = (P, hkv, PAGE_SIZE, d)
    if inv_freq is None:
        half = axes = 0
        pos_ptr = freq_ptr = pair = None
        if positions is not None or pair_axis is not None:
            raise ValueError("positions and pair_axis need inv_freq")
    else:
        half, axes = inv_freq.numel(), positions.shape[0]
        pos_ptr = _dense(positions, "positions", _I32, (axes, T), dev)
        freq_ptr = _dense(inv_freq, "inv_freq", _F32, (half,), dev)
        pair = _axes(pair_axis, half)
    st = (_lib or load_library()).k16v8_rope_kv_append_k8v8(
        q_ptr, q_ts, k.data_ptr(), _rows(k, "k", dt, row, dev), v.data_ptr(),
        _rows(v, "v", dt, row, dev), _X_DTYPES[dt],
        _dense(qo_indptr, "qo_indptr", _I32, (B + 1,), dev), T, pos_ptr, axes, pair, freq_ptr,
        2 * half, 1 if interleaved else 0, attn_factor,
        _dense(block_table, "block_table", _I32, (B, maxp), dev), maxp,
        _dense(seq_lens, "seq_lens", _I32, (B,), dev), B, out_ptr,
        _dense(k_cache, "k_cache", _U8, cache, dev), _dense(v_cache, "v_cache", _U8, cache, dev),
        _dense(kv_scale, "kv_scale", _F32, (P, hkv, 2), dev), P, hq, hkv, d,
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_rope_kv_append_k8v8", st)


def k16v8_decode_workspace_size_k8v8(batch, num_qo_heads, head_dim) -> int:
    """Bytes of workspace k16v8_paged_decode_attention_k8v8 needs on the current
    device (0 for an unsupported shape)."""
    return int(load_library().k16v8_decode_workspace_size_k8v8(batch, num_qo_heads, head_dim))


def _workspace(workspace, dev: int):
    """(address, bytes) of a dense workspace tensor."""
    if workspace is None:
        return None, 0
    return (_dense(workspace, "workspace", workspace.dtype, workspace.shape, dev),
            workspace.numel() * workspace.element_size())


def k16v8_paged_decode_attention_k8v8(q, k_cache, v_cache, kv_scale, block_table, seq_lens, sm_scale,
                                      workspace, out, lse=None, dev_error=None, stream=None) -> None:
    """Decode attention over the K8/V8 cache: q, out fp16 [B,Hq,D], lse fp32
    [B,Hq]; workspace uint8 of k16v8_decode_workspace_size_k8v8 bytes, not
    shared by calls that overlap."""
    B, hq, d = q.shape
    dev = _device(q)
    P, hkv = k_cache.shape[0], k_cache.shape[1]
    cache, maxp = (P, hkv, PAGE_SIZE, d), block_table.shape[1]
    ws, ws_bytes = _workspace(workspace, dev)
    st = (_lib or load_library()).k16v8_paged_decode_attention_k8v8(
        _dense(q, "q", _F16, (B, hq, d), dev), _dense(k_cache, "k_cache", _U8, cache, dev),
        _dense(v_cache, "v_cache", _U8, cache, dev),
        _dense(kv_scale, "kv_scale", _F32, (P, hkv, 2), dev),
        _dense(block_table, "block_table", _I32, (B, maxp), dev), maxp,
        _dense(seq_lens, "seq_lens", _I32, (B,), dev), B, hq, hkv, d, P, sm_scale, ws, ws_bytes,
        _dense(out, "out", _F16, (B, hq, d), dev),
        None if lse is None else _dense(lse, "lse", _F32, (B, hq), dev),
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error("k16v8_paged_decode_attention_k8v8", st)


def k16v8_attention_workspace_size_k8v8(max_qlen, num_qo_heads, num_kv_heads, head_dim) -> int:
    """Bytes of workspace the prefill and cross attention over the K8/V8 cache
    need on the current device (0 where the sizes are refused)."""
    return int(load_library().k16v8_attention_workspace_size_k8v8(max_qlen, num_qo_heads,
                                                                  num_kv_heads, head_dim))


def _attention_k8v8(name, q, qo_indptr, max_qlen, k_cache, v_cache, kv_scale, block_table, seq_lens,
                    max_seq_len, sm_scale, workspace, out, lse, dev_error, stream):
    total_q, hq, d = q.shape
    dev = _device(q)
    P, hkv = k_cache.shape[0], k_cache.shape[1]
    B, maxp = block_table.shape
    cache = (P, hkv, PAGE_SIZE, d)
    ws, ws_bytes = _workspace(workspace, dev)
    st = getattr(_lib or load_library(), name)(
        _dense(q, "q", _F16, (total_q, hq, d), dev),
        _dense(qo_indptr, "qo_indptr", _I32, (B + 1,), dev), total_q, max_qlen,
        _dense(k_cache, "k_cache", _U8, cache, dev), _dense(v_cache, "v_cache", _U8, cache, dev),
        _dense(kv_scale, "kv_scale", _F32, (P, hkv, 2), dev),
        _dense(block_table, "block_table", _I32, (B, maxp), dev), maxp,
        _dense(seq_lens, "seq_lens", _I32, (B,), dev), max_seq_len, B, hq, hkv, d, P, sm_scale, ws,
        ws_bytes, _dense(out, "out", _F16, (total_q, hq, d), dev),
        None if lse is None else _dense(lse, "lse", _F32, (total_q, hq), dev),
        _error_word(dev_error, dev), _stream_on(stream, dev))
    if st != K16V8_OK:
        raise K16V8Error(name, st)


def k16v8_paged_prefill_attention_k8v8(q, qo_indptr, max_qlen, k_cache, v_cache, kv_scale,
                                       block_table, seq_lens, max_seq_len, sm_scale, workspace, out,
                                       lse=None, dev_error=None, stream=None) -> None:
    """Causal attention of q fp16 [total_q,Hq,D] (ragged by qo_indptr int32
    [B+1]) over the K8/V8 cache, whose seq_lens include these tokens; at most
    max_qlen rows and max_seq_len positions per sequence; workspace uint8 of
    k16v8_attention_workspace_size_k8v8 bytes, not shared by calls that
    overlap."""
    _attention_k8v8("k16v8_paged_prefill_attention_k8v8", q, qo_indptr, max_qlen, k_cache, v_cache,
                    kv_scale, block_table, seq_lens, max_seq_len, sm_scale, workspace, out, lse,
                    dev_error, stream)


def k16v8_paged_cross_attention_k8v8(q, qo_indptr, max_qlen, k_cache, v_cache, kv_scale, block_table,
                                     seq_lens, max_seq_len, sm_scale, workspace, out, lse=None,
                                     dev_error=None, stream=None) -> None:
    """Attention of q fp16 [total_q,Hq,D] (ragged by qo_indptr int32 [B+1])
    over all seq_lens[b] positions of sequence b in the K8/V8 cache, e.g. an
    encoder's states; arguments as for the prefill call."""
    _attention_k8v8("k16v8_paged_cross_attention_k8v8", q, qo_indptr, max_qlen, k_cache, v_cache,
                    kv_scale, block_table, seq_lens, max_seq_len, sm_scale, workspace, out, lse,
                    dev_error, stream)


def k16v8_paged_prefill_attention_k8v8_wait_test(q, qo_indptr, max_qlen, k_cache, v_cache, kv_scale,
                                                 block_table, seq_lens, max_seq_len, sm_scale,
                                                 workspace, out, lse=None, dev_error=None,
                                                 stream=None) -> None:
    """Test hook: k16v8_paged_prefill_attention_k8v8 with the keys of the first
    CTA's first tile withheld, so that CTA's bounded wait expires
    (K16V8_DEVERR_TIMEOUT)."""
    _attention_k8v8("k16v8_paged_prefill_attention_k8v8_wait_test", q, qo_indptr, max_qlen, k_cache,
                    v_cache, kv_scale, block_table, seq_lens, max_seq_len, sm_scale, workspace, out,
                    lse, dev_error, stream)


def k16v8_read_device_error(dev_error, stream=None) -> int:
    """Synchronise the stream and return the device error word."""
    v = _i32()
    st = load_library().k16v8_read_device_error(_ptr(dev_error), _stream(stream),
                                                ctypes.byref(v))
    if st not in (K16V8_OK, K16V8_ERR_DEVICE_BOUNDS):
        _check("k16v8_read_device_error", st)
    return int(v.value)
