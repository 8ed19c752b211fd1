"""ctypes binding of ``libpaged_kv.so`` (the C ABI declared in ``include/pa.h``).

Argument marshalling only: tensors become device pointers and sizes, the current
torch stream becomes the ``void* stream`` argument, and a non-OK status becomes
an exception.  Every step of the computation runs in the library's kernels;
there is no fallback, and the import fails loudly if the library was not built.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpaged_kv.so")

PA_OK = 0
PA_F32, PA_BF16 = 0, 1
BLOCK_SIZE = 16
PARTITION_TOKENS = 512          # split-KV partition of pa_decode_attention at head_dim 128


def partition_tokens(head_dim: int) -> int:
    """Tokens per split-KV partition of pa_decode_attention (head_dim 64: twice as many)."""
    return 2 * PARTITION_TOKENS if head_dim == 64 else PARTITION_TOKENS

DEV_ERR_BAD_BLOCK = 1
DEV_ERR_BAD_POS = 2
DEV_ERR_HINT = 4
DEV_ERR_BAD_CU = 8
DEV_ERR_TIMEOUT = 16
DEV_ERR_BAD_PAIR = 32
DEV_ERR_BAD_PREFIX = 64

EXPORTED = [
    "pa_status_string", "pa_abi_version", "pa_append_kv", "pa_copy_block",
    "pa_decode_workspace_size", "pa_decode_attention", "pa_append_decode_attention",
    "pa_decode_attention_shared_prefix", "pa_append_decode_attention_shared_prefix",
    "pa_decode_attention_noalloc", "pa_append_kv_fp8", "pa_decode_attention_fp8",
    "pa_append_decode_attention_fp8",
    "pa_append_kv_fp4", "pa_decode_attention_fp4",
    "pa_prefill_attention", "pa_rope_append_kv", "pa_decode_attention_window",
    "pa_prefill_attention_window", "pa_rope_append_kv_axes", "pa_tree_workspace_size",
    "pa_tree_attention", "pa_compact_kv", "pa_bm_truncate", "pa_bm_create", "pa_bm_destroy",
    "pa_bm_add_seq", "pa_bm_fork", "pa_bm_free_seq", "pa_bm_blocks_needed",
    "pa_bm_prepare_append", "pa_bm_block_table", "pa_bm_block_tables", "pa_bm_seq_len",
    "pa_bm_refcount", "pa_bm_stats",
]


class PagedKVError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


class BmStats(ctypes.Structure):
    _fields_ = [("physical_blocks", ctypes.c_int64), ("free_blocks", ctypes.c_int64),
                ("logical_tokens", ctypes.c_int64), ("num_seqs", ctypes.c_int64)]


_lib = None
_quick = None                   # csrc/pa_binding.cpp, where it was built: see the bindings that use it


def lib() -> ctypes.CDLL:
    global _lib, _quick
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m paged_kv_cache_207_gb300.build` (nvcc, sm_103a)")
    L = ctypes.CDLL(_LIB_PATH)
    p, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    ip = ctypes.POINTER(ctypes.c_int32)
    L.pa_status_string.argtypes = [ctypes.c_int]
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_abi_version.restype = i32
    L.pa_append_kv.argtypes = [p, p, p, p, p, i32, p, p, i32, i32, i32, i32, i32, ctypes.c_int, p, p]
    L.pa_append_kv.restype = ctypes.c_int
    L.pa_copy_block.argtypes = [p, p, p, i32, i32, i32, i32, ctypes.c_int, p, p]
    L.pa_copy_block.restype = ctypes.c_int
    L.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.pa_decode_workspace_size.restype = sz
    L.pa_decode_attention.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32, i32,
                                      ctypes.c_float, ctypes.c_int, p, sz, p, p]
    L.pa_decode_attention.restype = ctypes.c_int
    L.pa_append_decode_attention.argtypes = [p, p, p, p, p, p, p, p, i32, i32, i32, i32, i32, i32,
                                             i32, ctypes.c_float, ctypes.c_int, p, sz, p, p]
    L.pa_append_decode_attention.restype = ctypes.c_int
    L.pa_decode_attention_shared_prefix.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32,
                                                    i32, ctypes.c_float, ctypes.c_int, i32, p, sz,
                                                    p, p]
    L.pa_decode_attention_shared_prefix.restype = ctypes.c_int
    L.pa_append_decode_attention_shared_prefix.argtypes = [p, p, p, p, p, p, p, p, i32, i32, i32,
                                                           i32, i32, i32, i32, ctypes.c_float,
                                                           ctypes.c_int, i32, p, sz, p, p]
    L.pa_append_decode_attention_shared_prefix.restype = ctypes.c_int
    L.pa_append_kv_fp8.argtypes = [p, p, p, p, p, i32, p, p, i32, i32, i32, i32, i32, p, p]
    L.pa_append_kv_fp8.restype = ctypes.c_int
    L.pa_decode_attention_fp8.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32, i32,
                                          ctypes.c_float, p, sz, p, p]
    L.pa_decode_attention_fp8.restype = ctypes.c_int
    L.pa_append_decode_attention_fp8.argtypes = [p, p, p, p, p, p, p, p, i32, i32, i32, i32, i32,
                                                 i32, i32, ctypes.c_float, p, sz, p, p]
    L.pa_append_decode_attention_fp8.restype = ctypes.c_int
    L.pa_append_kv_fp4.argtypes = [p, p, p, p, p, i32, p, p, i32, i32, i32, i32, i32, p, p]
    L.pa_append_kv_fp4.restype = ctypes.c_int
    L.pa_decode_attention_fp4.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32, i32,
                                          ctypes.c_float, p, sz, p, p]
    L.pa_decode_attention_fp4.restype = ctypes.c_int
    L.pa_prefill_attention.argtypes = [p, p, p, p, p, i32, p, p, i32, i32, i32, i32, i32, i32, i32,
                                       ctypes.c_float, ctypes.c_int, p, p]
    L.pa_prefill_attention.restype = ctypes.c_int
    i64 = ctypes.c_int64
    L.pa_rope_append_kv.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, p, i32, i32, p, i32, p, p,
                                    i32, i32, i32, i32, i32, i32, ctypes.c_int, p, p]
    L.pa_rope_append_kv.restype = ctypes.c_int
    L.pa_decode_attention_window.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32, i32, i32,
                                             ctypes.c_float, ctypes.c_int, p, p]
    L.pa_decode_attention_window.restype = ctypes.c_int
    L.pa_prefill_attention_window.argtypes = [p, p, p, p, p, i32, p, p, i32, i32, i32, i32, i32, i32,
                                              i32, i32, i32, ctypes.c_float, ctypes.c_int, p, p]
    L.pa_prefill_attention_window.restype = ctypes.c_int
    L.pa_rope_append_kv_axes.argtypes = [p, p, p, p, p, p, i64, i64, i64, i64, p, i32, i32, p, i32, p, p, i32, p,
                                         p, i32, i32, i32, i32, i32, i32, ctypes.c_int, p, p]
    L.pa_rope_append_kv_axes.restype = ctypes.c_int
    L.pa_tree_workspace_size.argtypes = [i32, i32, i32, i32]
    L.pa_tree_workspace_size.restype = sz
    L.pa_tree_attention.argtypes = [p, p, p, p, p, i32, p, p, p, i32, i32, i32, i32, i32, i32, i32, i32,
                                    ctypes.c_float, ctypes.c_int, p, sz, p, p]
    L.pa_tree_attention.restype = ctypes.c_int
    L.pa_compact_kv.argtypes = [p, p, p, i32, p, p, p, p, i32, i32, i32, i32, i32, i32, ctypes.c_int, p, p]
    L.pa_compact_kv.restype = ctypes.c_int
    L.pa_decode_attention_noalloc.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32, i32,
                                              ctypes.c_float, ctypes.c_int, p, p]
    L.pa_decode_attention_noalloc.restype = ctypes.c_int
    L.pa_bm_create.argtypes = [i32, ctypes.POINTER(p)]
    L.pa_bm_destroy.argtypes = [p]
    L.pa_bm_destroy.restype = None
    L.pa_bm_add_seq.argtypes = [p, ip]
    L.pa_bm_fork.argtypes = [p, i32, ip]
    L.pa_bm_free_seq.argtypes = [p, i32]
    L.pa_bm_blocks_needed.argtypes = [p, i32, i32, i32, ip]
    L.pa_bm_prepare_append.argtypes = [p, i32, i32, i32, ip, i32, ip]
    L.pa_bm_truncate.argtypes = [p, i32, i32]
    L.pa_bm_block_table.argtypes = [p, i32, ip, i32, ip]
    L.pa_bm_block_tables.argtypes = [p, ip, i32, ip, i32]
    L.pa_bm_seq_len.argtypes = [p, i32, ip]
    L.pa_bm_refcount.argtypes = [p, i32, ip]
    L.pa_bm_stats.argtypes = [p, ctypes.POINTER(BmStats)]
    for n in ("pa_bm_create", "pa_bm_add_seq", "pa_bm_fork", "pa_bm_free_seq",
              "pa_bm_blocks_needed", "pa_bm_prepare_append", "pa_bm_truncate", "pa_bm_block_table",
              "pa_bm_block_tables",
              "pa_bm_seq_len", "pa_bm_refcount", "pa_bm_stats"):
        getattr(L, n).restype = ctypes.c_int
    _lib = L
    try:
        from . import _quick as quick
    except ImportError:
        return L
    if quick.torch_version != torch.__version__:        # compiled for another torch: its tensors are laid out otherwise
        return L
    quick.bind(*(ctypes.cast(f, p).value for f in (L.pa_rope_append_kv, L.pa_decode_attention_window,
                                                   L.pa_prefill_attention_window, L.pa_rope_append_kv_axes,
                                                   L.pa_tree_attention, L.pa_compact_kv)))
    _quick = quick
    return L


def check(fn: str, status: int) -> None:
    if status != PA_OK:
        raise PagedKVError(fn, status, lib().pa_status_string(status).decode())


def _ptr(t) -> int:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor (device pointer)")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _i32(t, name):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    return _ptr(t)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.float32:
        return PA_F32
    raise TypeError(f"unsupported element type {t.dtype}")


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def pool_shape(num_blocks: int, num_kv_heads: int, head_dim: int, dtype: torch.dtype):
    """Shape of one K or V pool in the library's layout."""
    x = 16 // torch.empty((), dtype=dtype).element_size()
    return (num_blocks, num_kv_heads, head_dim // x, BLOCK_SIZE, x)


def fp8_pool_shape(num_blocks: int, num_kv_heads: int, head_dim: int):
    """Shape of one FP8 (E4M3) pool: per (block, kv head) a record of 16*D codes + 16 scales."""
    return (num_blocks, num_kv_heads, 16 * head_dim + 64)


def _fp8_dims(k_pool: torch.Tensor):
    if k_pool.dim() != 3 or k_pool.dtype != torch.uint8 or (k_pool.shape[2] - 64) % 16:
        raise ValueError("FP8 pools must be uint8 [num_blocks][Hkv][16*D + 64]")
    return k_pool.shape[0], k_pool.shape[1], (k_pool.shape[2] - 64) // 16


def append_kv_fp8(k_pool, v_pool, k_new, v_new, block_tables, start_pos, cu_new_tokens,
                  err_flag=None, stream=None) -> None:
    """Quantise bf16 rows ([tokens][Hkv][D]) into FP8 pools at explicit positions."""
    nb, hkv, d = _fp8_dims(k_pool)
    if k_new.dtype != torch.bfloat16 or v_new.dtype != torch.bfloat16:
        raise TypeError("new rows must be bf16")
    check("pa_append_kv_fp8", lib().pa_append_kv_fp8(
        _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new), _i32(block_tables, "block_tables"),
        block_tables.shape[1], _i32(start_pos, "start_pos"), _i32(cu_new_tokens, "cu_new_tokens"),
        start_pos.shape[0], k_new.shape[0], nb, hkv, d,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def decode_attention_fp8(out, q, k_pool, v_pool, block_tables, context_lens, scale, workspace=None,
                         max_context_len_hint: int = 0, err_flag=None, stream=None) -> None:
    """decode_attention over FP8 pools (bf16 q and out)."""
    nb, hkv, d = _fp8_dims(k_pool)
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("q and out must be bf16")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention_fp8", lib().pa_decode_attention_fp8(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _i32(block_tables, "block_tables"),
        _i32(context_lens, "context_lens"), q.shape[0], q.shape[1], hkv, d, block_tables.shape[1],
        int(max_context_len_hint), nb, float(scale),
        None if workspace is None else _ptr(workspace), ws_bytes,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def append_decode_attention_fp8(out, q, k_pool, v_pool, k_new, v_new, block_tables, context_lens,
                                scale, workspace=None, max_context_len_hint: int = 0,
                                err_flag=None, stream=None) -> None:
    """decode_attention_fp8 with the step's bf16 rows k_new / v_new ([S][Hkv][D]) quantised
    and written at position context_lens[s] - 1 by the decode kernel itself."""
    nb, hkv, d = _fp8_dims(k_pool)
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("q and out must be bf16")
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        if tuple(t.shape) != (q.shape[0], hkv, d) or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 [num_seqs][num_kv_heads][head_dim] tensor")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_append_decode_attention_fp8", lib().pa_append_decode_attention_fp8(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new),
        _i32(block_tables, "block_tables"), _i32(context_lens, "context_lens"), q.shape[0],
        q.shape[1], hkv, d, block_tables.shape[1], int(max_context_len_hint), nb, float(scale),
        None if workspace is None else _ptr(workspace), ws_bytes,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def copy_block_fp8(k_pool, v_pool, pairs, err_flag=None, stream=None) -> None:
    """copy_block for FP8 pools."""
    nb, hkv, d = _fp8_dims(k_pool)
    check("pa_copy_block", lib().pa_copy_block(
        _ptr(k_pool), _ptr(v_pool), _i32(pairs, "pairs"), pairs.shape[0], nb, hkv, d, 2,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def fp4_pool_shape(num_blocks: int, num_kv_heads: int, head_dim: int):
    """Shape of one MXFP4 pool: per (block, kv head) 8*D code bytes + D/2 scale bytes."""
    return (num_blocks, num_kv_heads, 8 * head_dim + head_dim // 2)


def _fp4_dims(k_pool: torch.Tensor):
    if k_pool.dim() != 3 or k_pool.dtype != torch.uint8 or k_pool.shape[2] % 17:
        raise ValueError("FP4 pools must be uint8 [num_blocks][Hkv][8*D + D/2]")
    return k_pool.shape[0], k_pool.shape[1], k_pool.shape[2] * 2 // 17


def append_kv_fp4(k_pool, v_pool, k_new, v_new, block_tables, start_pos, cu_new_tokens,
                  err_flag=None, stream=None) -> None:
    """Quantise bf16 rows ([tokens][Hkv][D]) into MXFP4 pools at explicit positions."""
    nb, hkv, d = _fp4_dims(k_pool)
    if k_new.dtype != torch.bfloat16 or v_new.dtype != torch.bfloat16:
        raise TypeError("new rows must be bf16")
    check("pa_append_kv_fp4", lib().pa_append_kv_fp4(
        _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new), _i32(block_tables, "block_tables"),
        block_tables.shape[1], _i32(start_pos, "start_pos"), _i32(cu_new_tokens, "cu_new_tokens"),
        start_pos.shape[0], k_new.shape[0], nb, hkv, d,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def decode_attention_fp4(out, q, k_pool, v_pool, block_tables, context_lens, scale, workspace=None,
                         max_context_len_hint: int = 0, err_flag=None, stream=None) -> None:
    """decode_attention over MXFP4 pools (bf16 q and out)."""
    nb, hkv, d = _fp4_dims(k_pool)
    if q.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("q and out must be bf16")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention_fp4", lib().pa_decode_attention_fp4(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _i32(block_tables, "block_tables"),
        _i32(context_lens, "context_lens"), q.shape[0], q.shape[1], hkv, d, block_tables.shape[1],
        int(max_context_len_hint), nb, float(scale),
        None if workspace is None else _ptr(workspace), ws_bytes,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def copy_block_fp4(k_pool, v_pool, pairs, err_flag=None, stream=None) -> None:
    """copy_block for MXFP4 pools."""
    nb, hkv, d = _fp4_dims(k_pool)
    check("pa_copy_block", lib().pa_copy_block(
        _ptr(k_pool), _ptr(v_pool), _i32(pairs, "pairs"), pairs.shape[0], nb, hkv, d, 3,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def _pool_dims(k_pool: torch.Tensor):
    if k_pool.dim() != 5 or k_pool.shape[3] != BLOCK_SIZE:
        raise ValueError("pools must have shape [num_blocks][Hkv][D/X][16][X]")
    return k_pool.shape[0], k_pool.shape[1], k_pool.shape[2] * k_pool.shape[4]


def append_kv(k_pool, v_pool, k_new, v_new, block_tables, start_pos, cu_new_tokens,
              err_flag=None, stream=None) -> None:
    """Write rows of k_new / v_new ([tokens][Hkv][D]) at explicit positions."""
    nb, hkv, d = _pool_dims(k_pool)
    check("pa_append_kv", lib().pa_append_kv(
        _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new), _i32(block_tables, "block_tables"),
        block_tables.shape[1], _i32(start_pos, "start_pos"), _i32(cu_new_tokens, "cu_new_tokens"),
        start_pos.shape[0], k_new.shape[0], nb, hkv, d, _dtype_code(k_pool),
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def copy_block(k_pool, v_pool, pairs, err_flag=None, stream=None) -> None:
    """Copy whole blocks src -> dst (pairs: int32 [n][2] on the device)."""
    nb, hkv, d = _pool_dims(k_pool)
    check("pa_copy_block", lib().pa_copy_block(
        _ptr(k_pool), _ptr(v_pool), _i32(pairs, "pairs"), pairs.shape[0], nb, hkv, d,
        _dtype_code(k_pool), None if err_flag is None else _i32(err_flag, "err_flag"),
        _stream(stream)))


def decode_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                          max_blocks_per_seq: int) -> int:
    return int(lib().pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                              max_blocks_per_seq))


def decode_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                     max_blocks_per_seq: int, device="cuda"):
    """A zero-filled workspace for decode_attention (None when none is needed)."""
    n = decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def decode_attention(out, q, k_pool, v_pool, block_tables, context_lens, scale, workspace=None,
                     max_context_len_hint: int = 0, err_flag=None, stream=None) -> None:
    """Single-token attention of q ([S][Hq][D]) over the paged cache into out."""
    nb, hkv, d = _pool_dims(k_pool)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention", lib().pa_decode_attention(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _i32(block_tables, "block_tables"),
        _i32(context_lens, "context_lens"), q.shape[0], q.shape[1], hkv, d, block_tables.shape[1],
        int(max_context_len_hint), nb, float(scale), _dtype_code(q),
        None if workspace is None else _ptr(workspace), ws_bytes,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def append_decode_attention(out, q, k_pool, v_pool, k_new, v_new, block_tables, context_lens,
                            scale, workspace=None, max_context_len_hint: int = 0, err_flag=None,
                            stream=None) -> None:
    """One decode step in one call: k_new / v_new ([S][Hkv][D]) go to position
    context_lens[s] - 1 (context_lens counts the new token), then decode_attention."""
    nb, hkv, d = _pool_dims(k_pool)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        if tuple(t.shape) != (q.shape[0], hkv, d) or t.dtype != k_pool.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [num_seqs][num_kv_heads][head_dim] "
                             f"tensor of the pool's type")
    check("pa_append_decode_attention", lib().pa_append_decode_attention(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new),
        _i32(block_tables, "block_tables"), _i32(context_lens, "context_lens"), q.shape[0],
        q.shape[1], hkv, d, block_tables.shape[1], int(max_context_len_hint), nb, float(scale),
        _dtype_code(q), None if workspace is None else _ptr(workspace), ws_bytes,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def append_decode_attention_shared_prefix(out, q, k_pool, v_pool, k_new, v_new, block_tables,
                                          context_lens, scale, shared_prefix_tokens: int,
                                          workspace=None, max_context_len_hint: int = 0,
                                          err_flag=None, stream=None) -> None:
    """decode_attention_shared_prefix with the step's new rows written by the decode kernel
    (k_new / v_new [S][Hkv][D] go to position context_lens[s] - 1, past the prefix)."""
    nb, hkv, d = _pool_dims(k_pool)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    for t, name in ((k_new, "k_new"), (v_new, "v_new")):
        if tuple(t.shape) != (q.shape[0], hkv, d) or t.dtype != k_pool.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [num_seqs][num_kv_heads][head_dim] "
                             f"tensor of the pool's type")
    check("pa_append_decode_attention_shared_prefix", lib().pa_append_decode_attention_shared_prefix(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new),
        _i32(block_tables, "block_tables"), _i32(context_lens, "context_lens"), q.shape[0],
        q.shape[1], hkv, d, block_tables.shape[1], int(max_context_len_hint), nb, float(scale),
        _dtype_code(q), int(shared_prefix_tokens), None if workspace is None else _ptr(workspace),
        ws_bytes, None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def decode_attention_shared_prefix(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                                   shared_prefix_tokens: int, workspace=None,
                                   max_context_len_hint: int = 0, err_flag=None,
                                   stream=None) -> None:
    """decode_attention for a batch whose sequences share their first
    ``shared_prefix_tokens`` positions in the same physical blocks."""
    nb, hkv, d = _pool_dims(k_pool)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention_shared_prefix", lib().pa_decode_attention_shared_prefix(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _i32(block_tables, "block_tables"),
        _i32(context_lens, "context_lens"), q.shape[0], q.shape[1], hkv, d, block_tables.shape[1],
        int(max_context_len_hint), nb, float(scale), _dtype_code(q), int(shared_prefix_tokens),
        None if workspace is None else _ptr(workspace), ws_bytes,
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


def prefill_attention(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, scale,
                      max_chunk: int, err_flag=None, stream=None) -> None:
    """Causal attention of chunk rows q ([total][Hq][D]) over the paged cache."""
    nb, hkv, d = _pool_dims(k_pool)
    check("pa_prefill_attention", lib().pa_prefill_attention(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _i32(block_tables, "block_tables"),
        block_tables.shape[1], _i32(start_pos, "start_pos"), _i32(cu_q, "cu_q"),
        start_pos.shape[0], q.shape[0], int(max_chunk), q.shape[1], hkv, d, nb, float(scale),
        _dtype_code(q), None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


# Bindings of the rotary append and of the windowed attention.  A decode step calls them once per
# layer, and a short step waits for them rather than for the GPU: a call whose arguments are all
# as they should be, on the current device and stream, goes through csrc/pa_binding.cpp, which
# makes the same checks.  Where that answers -1 (or was not built), the tensors are checked here,
# in one expression, and only when it is false each is looked at again for the reason.
_PLAIN_CODE = {torch.float32: PA_F32, torch.bfloat16: PA_BF16}
_I32 = torch.int32
_cuda_device = torch.cuda.current_device


def _plain_pool(k_pool):
    """Blocks, kv heads, head_dim, pool code and the type of rows, q and out."""
    try:
        nb, hkv, pieces, slots, x = k_pool.shape
    except ValueError:
        slots = 0
    if slots != BLOCK_SIZE:
        raise ValueError("pools must have shape [num_blocks][Hkv][D/X][16][X]")
    dtype = k_pool.dtype
    code = _PLAIN_CODE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported element type {dtype}")
    return nb, hkv, pieces * x, code, dtype


def _fp8_pool(k_pool):
    return *_fp8_dims(k_pool), 2, torch.bfloat16


def _fp4_pool(k_pool):
    return *_fp4_dims(k_pool), 3, torch.bfloat16


def _bound(x) -> int:
    """A window, sink count or chunk bound as an int32: anything past its ends is as good as the
    end (ctypes would take it modulo 2^32)."""
    return max(-2**31, min(int(x), 2**31 - 1))


def _call_on(dev: int, stream, fn, *args) -> None:
    """Calls a library function on device `dev`, on its current stream by default."""
    if dev != _cuda_device():
        with torch.cuda.device(dev):
            return _call_on(dev, stream, fn, *args)
    # (the raw handle: building a Stream object costs as much as the launch)
    status = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status != PA_OK:
        check(fn.__name__, status)


def _refuse(dev, t, name, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the pools' device")
    raise ValueError(f"{name} must be contiguous")


def _checked(dev, t, name, dtype, shape):
    """Address of a contiguous tensor of this device (an index), type and shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev >= 0 and t.is_contiguous()):
        _refuse(dev, t, name, dtype, shape)
    return t.data_ptr()


def _rows(dev, t, name, dtype, shape):
    """Address and row stride of rows [n][heads][head_dim] whose rows may lie apart."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev >= 0):
        _refuse(dev, t, name, dtype, shape)
    row, head, one = t.stride()
    n, heads, d = shape
    if n and (one != 1 or (heads > 1 and head != d)):
        raise ValueError(f"{name}: a row's heads must be contiguous")
    return t.data_ptr(), (row if n > 1 else heads * d)


def _flag(dev, err_flag):
    return None if err_flag is None else _checked(dev, err_flag, "err_flag", _I32, err_flag.shape)


def _rope_append(pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos,
                 cu_new_tokens, interleaved, err_flag, stream, axes=None) -> None:
    nb, hkv, d, code, rows = pool(k_pool)
    if q is None or q_out is None:
        if q is not q_out:
            raise ValueError("q and q_out come together")
        q = q_out = k_new                               # (checked once more, not used)
        with_q = False
    else:
        with_q = True
    try:
        dev, shape, kind = k_pool.get_device(), k_pool.shape, k_pool.dtype
        (half,) = inv_freq.shape
        s, width = block_tables.shape
        n, hq, _ = of_q = q.shape
        of_k = (n, hkv, d)
        q_row, q_head, q_one = q.stride()
        o_row, o_head, o_one = q_out.stride()
        k_row, k_head, k_one = k_new.stride()
        v_row, v_head, v_one = v_new.stride()
        fine = (q.dtype is rows and q_out.dtype is rows and k_new.dtype is rows and v_new.dtype is rows
                and of_q[2] == d and q_out.shape == of_q and k_new.shape == of_k and v_new.shape == of_k
                and q_one == o_one == k_one == v_one == 1 and q_head == o_head == k_head == v_head == d
                and v_pool.dtype is kind and v_pool.shape == shape and inv_freq.dtype is torch.float64
                and block_tables.dtype is _I32 and start_pos.dtype is _I32 and cu_new_tokens.dtype is _I32
                and start_pos.shape == (s,) and cu_new_tokens.shape == (s + 1,)
                and q.get_device() == q_out.get_device() == k_new.get_device() == v_new.get_device()
                == v_pool.get_device() == inv_freq.get_device() == block_tables.get_device()
                == start_pos.get_device() == cu_new_tokens.get_device() == dev >= 0
                and k_pool.is_contiguous() and v_pool.is_contiguous() and inv_freq.is_contiguous()
                and block_tables.is_contiguous() and start_pos.is_contiguous() and cu_new_tokens.is_contiguous())
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        # one by one, for the reason (or none: a single head's stride, or no rows, say nothing)
        dev, shape, kind = k_pool.get_device(), k_pool.shape, k_pool.dtype
        n = k_new.shape[0]
        _, k_row = _rows(dev, k_new, "k_new", rows, (n, hkv, d))
        _, v_row = _rows(dev, v_new, "v_new", rows, (n, hkv, d))
        hq = q.shape[1]
        _, q_row = _rows(dev, q, "q", rows, (n, hq, d))
        _, o_row = _rows(dev, q_out, "q_out", rows, (n, hq, d))
        s, width, half = block_tables.shape[0], block_tables.shape[1], inv_freq.shape[0]
        _checked(dev, k_pool, "k_pool", kind, shape)
        _checked(dev, v_pool, "v_pool", kind, shape)
        _checked(dev, inv_freq, "inv_freq", torch.float64, (half,))
        _checked(dev, block_tables, "block_tables", _I32, (s, width))
        _checked(dev, start_pos, "start_pos", _I32, (s,))
        _checked(dev, cu_new_tokens, "cu_new_tokens", _I32, (s + 1,))
    fn, more = lib().pa_rope_append_kv, ()
    if axes is not None:
        plane_axis, positions = axes
        if not isinstance(positions, torch.Tensor) or positions.dim() != 2 or positions.shape[0] < 1:
            raise ValueError("positions must be an int32 [axes][tokens] tensor")
        num = positions.shape[0]
        at = _checked(dev, positions, "positions", _I32, (num, n))
        if plane_axis is None and num > 1:
            raise ValueError("plane_axis must name the axis of each plane where there are several")
        fn, more = lib().pa_rope_append_kv_axes, (
            at, num, None if plane_axis is None else _checked(dev, plane_axis, "plane_axis", _I32, (half,)))
    _call_on(dev, stream, fn, k_pool.data_ptr(), v_pool.data_ptr(),
             q_out.data_ptr() if with_q else None, q.data_ptr() if with_q else None, k_new.data_ptr(),
             v_new.data_ptr(), o_row, q_row, k_row, v_row, inv_freq.data_ptr(), _bound(2 * half),
             1 if interleaved else 0, *more, block_tables.data_ptr(), width, start_pos.data_ptr(),
             cu_new_tokens.data_ptr(), s, n, nb, hq if with_q else 0, hkv, d, code,
             None if err_flag is None else _flag(dev, err_flag))


def rope_append_kv(k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos,
                   cu_new_tokens, interleaved: bool = False, err_flag=None, stream=None) -> None:
    """append_kv with the position rotation on the way: queries and keys of row i of sequence s
    are turned by (start_pos[s] + i) * inv_freq (float64 [rotary_dim / 2] on the device), keys
    and values go to the pools, the turned queries to q_out (which may be q; both None: no
    queries).  Rows [tokens][heads][D] may be column ranges of a wider tensor."""
    status = -1 if _quick is None else _quick.rope_append(
        0, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos, cu_new_tokens,
        interleaved, err_flag, stream)
    if status == -1:
        _rope_append(_plain_pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables,
                     start_pos, cu_new_tokens, interleaved, err_flag, stream)
    elif status:
        check("pa_rope_append_kv", status)


def rope_append_kv_fp8(k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos,
                       cu_new_tokens, interleaved: bool = False, err_flag=None, stream=None) -> None:
    """rope_append_kv of bf16 rows into FP8 pools."""
    status = -1 if _quick is None else _quick.rope_append(
        2, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos, cu_new_tokens,
        interleaved, err_flag, stream)
    if status == -1:
        _rope_append(_fp8_pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables,
                     start_pos, cu_new_tokens, interleaved, err_flag, stream)
    elif status:
        check("pa_rope_append_kv", status)


def rope_append_kv_fp4(k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos,
                       cu_new_tokens, interleaved: bool = False, err_flag=None, stream=None) -> None:
    """rope_append_kv of bf16 rows into MXFP4 pools."""
    status = -1 if _quick is None else _quick.rope_append(
        3, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos, cu_new_tokens,
        interleaved, err_flag, stream)
    if status == -1:
        _rope_append(_fp4_pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables,
                     start_pos, cu_new_tokens, interleaved, err_flag, stream)
    elif status:
        check("pa_rope_append_kv", status)


def _rope_axes(kind, pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
               start_pos, cu_new_tokens, interleaved, err_flag, stream) -> None:
    status = -1 if _quick is None else _quick.rope_axes(
        kind, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables, start_pos,
        cu_new_tokens, interleaved, err_flag, stream)
    if status == -1:
        _rope_append(pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, block_tables, start_pos, cu_new_tokens,
                     interleaved, err_flag, stream, (plane_axis, positions))
    elif status:
        check("pa_rope_append_kv_axes", status)


def rope_append_kv_axes(k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
                        start_pos, cu_new_tokens, interleaved: bool = False, err_flag=None, stream=None) -> None:
    """rope_append_kv whose rows are turned by positions of their own: plane f of row r by
    positions[plane_axis[f], r] * inv_freq[f] (positions int32 [axes][tokens], plane_axis int32
    [rotary_dim / 2], None for a single axis).  A drafted tree's nodes turn by their depth (one
    axis), an image's tokens by time, height and width (three)."""
    _rope_axes(0, _plain_pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
               start_pos, cu_new_tokens, interleaved, err_flag, stream)


def rope_append_kv_axes_fp8(k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
                            start_pos, cu_new_tokens, interleaved: bool = False, err_flag=None, stream=None) -> None:
    """rope_append_kv_axes of bf16 rows into FP8 pools."""
    _rope_axes(2, _fp8_pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
               start_pos, cu_new_tokens, interleaved, err_flag, stream)


def rope_append_kv_axes_fp4(k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
                            start_pos, cu_new_tokens, interleaved: bool = False, err_flag=None, stream=None) -> None:
    """rope_append_kv_axes of bf16 rows into MXFP4 pools."""
    _rope_axes(3, _fp4_pool, k_pool, v_pool, q_out, q, k_new, v_new, inv_freq, plane_axis, positions, block_tables,
               start_pos, cu_new_tokens, interleaved, err_flag, stream)


def tree_workspace_size(num_q_heads: int, num_kv_heads: int, head_dim: int, max_chunk: int) -> int:
    return int(lib().pa_tree_workspace_size(num_q_heads, num_kv_heads, head_dim, _bound(max_chunk)))


def tree_workspace(num_q_heads: int, num_kv_heads: int, head_dim: int, max_chunk: int, device="cuda"):
    """A workspace for tree_attention of trees of at most max_chunk nodes."""
    return torch.empty(tree_workspace_size(num_q_heads, num_kv_heads, head_dim, max_chunk), dtype=torch.uint8, device=device)


def _tree(kind, pool, out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk, workspace,
          err_flag, stream) -> None:
    status = -1 if _quick is None else _quick.tree(
        kind, out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk, workspace, err_flag,
        stream)
    if status > 0:
        check("pa_tree_attention", status)
    if status != -1:
        return
    nb, hkv, d, code, rows = pool(k_pool)
    dev = k_pool.get_device()
    for t, name, dims in ((block_tables, "block_tables", 2), (q, "q", 3), (tree_mask, "tree_mask", 2)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a tensor of {dims} dimensions")
    (s, width), (n, hq, _), words = block_tables.shape, q.shape, tree_mask.shape[1]
    for t, name, dtype, of_t in ((q, "q", rows, (n, hq, d)), (out, "out", rows, (n, hq, d)),
                                 (k_pool, "k_pool", k_pool.dtype, k_pool.shape),
                                 (v_pool, "v_pool", k_pool.dtype, k_pool.shape),
                                 (block_tables, "block_tables", _I32, (s, width)), (start_pos, "start_pos", _I32, (s,)),
                                 (cu_q, "cu_q", _I32, (s + 1,)), (tree_mask, "tree_mask", _I32, (n, words))):
        _checked(dev, t, name, dtype, of_t)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch tensor (see tree_workspace)")
    _checked(dev, workspace, "workspace", workspace.dtype, workspace.shape)
    _call_on(dev, stream, lib().pa_tree_attention, out.data_ptr(), q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
             block_tables.data_ptr(), width, start_pos.data_ptr(), cu_q.data_ptr(), tree_mask.data_ptr(), words, s, n,
             _bound(max_chunk), hq, hkv, d, nb, float(scale), code, workspace.data_ptr(),
             workspace.numel() * workspace.element_size(), None if err_flag is None else _flag(dev, err_flag))


def tree_attention(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk: int, workspace,
                   err_flag=None, stream=None) -> None:
    """Attention of drafted trees: row cu_q[s] + i of q ([total][Hq][D]), node i of sequence s at
    position start_pos[s] + i, sees the positions before start_pos[s] and the nodes j whose bit
    (j % 32 of word j / 32) its row of tree_mask (int32 [total][words]) sets.  No tree has more than
    max_chunk nodes; workspace: see tree_workspace."""
    _tree(0, _plain_pool, out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk, workspace,
          err_flag, stream)


def tree_attention_fp8(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk: int, workspace,
                       err_flag=None, stream=None) -> None:
    """tree_attention over FP8 pools (bf16 q and out)."""
    _tree(2, _fp8_pool, out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk, workspace,
          err_flag, stream)


def tree_attention_fp4(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk: int, workspace,
                       err_flag=None, stream=None) -> None:
    """tree_attention over MXFP4 pools (bf16 q and out)."""
    _tree(3, _fp4_pool, out, q, k_pool, v_pool, block_tables, start_pos, cu_q, tree_mask, scale, max_chunk, workspace,
          err_flag, stream)


def _compact(kind, pool, k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables, err_flag, stream) -> None:
    status = -1 if _quick is None else _quick.compact(
        kind, k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables, err_flag, stream)
    if status > 0:
        check("pa_compact_kv", status)
    if status != -1:
        return
    nb, hkv, d, code, _ = pool(k_pool)
    dev = k_pool.get_device()
    for t, name, dims in ((block_tables, "block_tables", 2), (src_pos, "src_pos", 1)) + (
            () if dst_tables is None else ((dst_tables, "dst_tables", 2),)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a tensor of {dims} dimensions")
    (s, width), n = block_tables.shape, src_pos.shape[0]
    if dst_tables is not None and dst_tables.shape[1] == 0 and n > 0:
        raise ValueError("dst_tables has no columns")        # (its address, null, would mean in place)
    for t, name, dtype, of_t in ((k_pool, "k_pool", k_pool.dtype, k_pool.shape),
                                 (v_pool, "v_pool", k_pool.dtype, k_pool.shape),
                                 (block_tables, "block_tables", _I32, (s, width)), (src_pos, "src_pos", _I32, (n,)),
                                 (dst_start, "dst_start", _I32, (s,)), (cu_rows, "cu_rows", _I32, (s + 1,))):
        _checked(dev, t, name, dtype, of_t)
    to = (None, 0) if dst_tables is None else (
        _checked(dev, dst_tables, "dst_tables", _I32, (s, dst_tables.shape[1])), dst_tables.shape[1])
    _call_on(dev, stream, lib().pa_compact_kv, k_pool.data_ptr(), v_pool.data_ptr(), block_tables.data_ptr(), width,
             src_pos.data_ptr(), dst_start.data_ptr(), cu_rows.data_ptr(), *to, s, n, nb, hkv, d, code,
             None if err_flag is None else _flag(dev, err_flag))


def compact_kv(k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables=None, err_flag=None,
               stream=None) -> None:
    """Moves rows to consecutive positions: row i of sequence s from position
    src_pos[cu_rows[s] + i] to dst_start[s] + i.  In place (dst_tables None) a row may not come from
    before its destination; with dst_tables ([num_seqs][width]) the rows go to blocks that are none
    of the sources', in any order.  cu_rows may end below src_pos's length."""
    _compact(0, _plain_pool, k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables, err_flag, stream)


def compact_kv_fp8(k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables=None, err_flag=None,
                   stream=None) -> None:
    """compact_kv for FP8 pools."""
    _compact(2, _fp8_pool, k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables, err_flag, stream)


def compact_kv_fp4(k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables=None, err_flag=None,
                   stream=None) -> None:
    """compact_kv for MXFP4 pools."""
    _compact(3, _fp4_pool, k_pool, v_pool, block_tables, src_pos, dst_start, cu_rows, dst_tables, err_flag, stream)


def _decode_window(pool, out, q, k_pool, v_pool, block_tables, context_lens, scale, window, num_sinks,
                   err_flag, stream) -> None:
    nb, hkv, d, code, rows = pool(k_pool)
    try:
        dev, shape, kind = k_pool.get_device(), k_pool.shape, k_pool.dtype
        s, width = block_tables.shape
        n, hq, dq = of_q = q.shape
        fine = (n == s and dq == d and q.dtype is rows and out.dtype is rows and out.shape == of_q
                and v_pool.dtype is kind and v_pool.shape == shape and block_tables.dtype is _I32
                and context_lens.dtype is _I32 and context_lens.shape == (s,)
                and q.get_device() == out.get_device() == v_pool.get_device() == block_tables.get_device()
                == context_lens.get_device() == dev >= 0
                and q.is_contiguous() and out.is_contiguous() and k_pool.is_contiguous()
                and v_pool.is_contiguous() and block_tables.is_contiguous() and context_lens.is_contiguous())
    except (AttributeError, ValueError):
        fine = False
    if not fine:                                        # one by one, for the reason
        s, width = block_tables.shape[0], block_tables.shape[1]
        hq = q.shape[1]
        for t, name, dtype, of_t in ((q, "q", rows, (s, hq, d)), (out, "out", rows, (s, hq, d)),
                                     (k_pool, "k_pool", k_pool.dtype, k_pool.shape),
                                     (v_pool, "v_pool", k_pool.dtype, k_pool.shape),
                                     (block_tables, "block_tables", _I32, (s, width)),
                                     (context_lens, "context_lens", _I32, (s,))):
            _checked(k_pool.get_device(), t, name, dtype, of_t)
        raise ValueError("arguments of different shapes, types or devices")
    _call_on(dev, stream, lib().pa_decode_attention_window, out.data_ptr(), q.data_ptr(), k_pool.data_ptr(),
             v_pool.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), s, hq, hkv, d, width, nb,
             _bound(window), _bound(num_sinks), float(scale), code,
             None if err_flag is None else _flag(dev, err_flag))


def decode_attention_window(out, q, k_pool, v_pool, block_tables, context_lens, scale, window: int,
                            num_sinks: int = 0, err_flag=None, stream=None) -> None:
    """decode_attention over the last ``window`` positions and the first ``num_sinks``; table
    entries of blocks that hold none of them are not read."""
    status = -1 if _quick is None else _quick.decode_window(
        0, out, q, k_pool, v_pool, block_tables, context_lens, scale, window, num_sinks, err_flag, stream)
    if status == -1:
        _decode_window(_plain_pool, out, q, k_pool, v_pool, block_tables, context_lens, scale, window,
                       num_sinks, err_flag, stream)
    elif status:
        check("pa_decode_attention_window", status)


def decode_attention_window_fp8(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                                window: int, num_sinks: int = 0, err_flag=None, stream=None) -> None:
    """decode_attention_window over FP8 pools (bf16 q and out)."""
    status = -1 if _quick is None else _quick.decode_window(
        2, out, q, k_pool, v_pool, block_tables, context_lens, scale, window, num_sinks, err_flag, stream)
    if status == -1:
        _decode_window(_fp8_pool, out, q, k_pool, v_pool, block_tables, context_lens, scale, window,
                       num_sinks, err_flag, stream)
    elif status:
        check("pa_decode_attention_window", status)


def decode_attention_window_fp4(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                                window: int, num_sinks: int = 0, err_flag=None, stream=None) -> None:
    """decode_attention_window over MXFP4 pools (bf16 q and out)."""
    status = -1 if _quick is None else _quick.decode_window(
        3, out, q, k_pool, v_pool, block_tables, context_lens, scale, window, num_sinks, err_flag, stream)
    if status == -1:
        _decode_window(_fp4_pool, out, q, k_pool, v_pool, block_tables, context_lens, scale, window,
                       num_sinks, err_flag, stream)
    elif status:
        check("pa_decode_attention_window", status)


def prefill_attention_window(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, scale,
                             max_chunk: int, window: int, num_sinks: int = 0, err_flag=None,
                             stream=None) -> None:
    """prefill_attention with every row limited to the last ``window`` positions up to its own
    and the first ``num_sinks`` (bf16)."""
    status = -1 if _quick is None else _quick.prefill_window(
        out, q, k_pool, v_pool, block_tables, start_pos, cu_q, scale, max_chunk, window, num_sinks, err_flag,
        stream)
    if status == -1:
        _prefill_window(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, scale, max_chunk, window,
                        num_sinks, err_flag, stream)
    elif status:
        check("pa_prefill_attention_window", status)


def _prefill_window(out, q, k_pool, v_pool, block_tables, start_pos, cu_q, scale, max_chunk, window,
                    num_sinks, err_flag, stream) -> None:
    nb, hkv, d, code, rows = _plain_pool(k_pool)
    try:
        dev, shape, kind = k_pool.get_device(), k_pool.shape, k_pool.dtype
        s, width = block_tables.shape
        n, hq, dq = of_q = q.shape
        fine = (dq == d and q.dtype is rows and out.dtype is rows and out.shape == of_q
                and v_pool.dtype is kind and v_pool.shape == shape and block_tables.dtype is _I32
                and start_pos.dtype is _I32 and start_pos.shape == (s,)
                and cu_q.dtype is _I32 and cu_q.shape == (s + 1,)
                and q.get_device() == out.get_device() == v_pool.get_device() == block_tables.get_device()
                == start_pos.get_device() == cu_q.get_device() == dev >= 0
                and q.is_contiguous() and out.is_contiguous() and k_pool.is_contiguous()
                and v_pool.is_contiguous() and block_tables.is_contiguous() and start_pos.is_contiguous()
                and cu_q.is_contiguous())
    except (AttributeError, ValueError):
        fine = False
    if not fine:                                        # one by one, for the reason
        s, width = block_tables.shape[0], block_tables.shape[1]
        n, hq = q.shape[0], q.shape[1]
        for t, name, dtype, of_t in ((q, "q", rows, (n, hq, d)), (out, "out", rows, (n, hq, d)),
                                     (k_pool, "k_pool", k_pool.dtype, k_pool.shape),
                                     (v_pool, "v_pool", k_pool.dtype, k_pool.shape),
                                     (block_tables, "block_tables", _I32, (s, width)),
                                     (start_pos, "start_pos", _I32, (s,)), (cu_q, "cu_q", _I32, (s + 1,))):
            _checked(k_pool.get_device(), t, name, dtype, of_t)
        raise ValueError("arguments of different shapes, types or devices")
    _call_on(dev, stream, lib().pa_prefill_attention_window, out.data_ptr(), q.data_ptr(), k_pool.data_ptr(),
             v_pool.data_ptr(), block_tables.data_ptr(), width, start_pos.data_ptr(), cu_q.data_ptr(), s, n,
             _bound(max_chunk), hq, hkv, d, nb, _bound(window), _bound(num_sinks), float(scale), code,
             None if err_flag is None else _flag(dev, err_flag))


NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024
PA_ERR_SCRATCH_LIMIT = 5


def decode_attention_noalloc(out, q, k_pool, v_pool, block_tables, context_lens, scale,
                             max_context_len_hint: int = 0, err_flag=None, stream=None) -> None:
    """decode_attention without a caller workspace: the library's built-in 16 MiB device
    scratch is used instead (for callers that cannot allocate device memory)."""
    nb, hkv, d = _pool_dims(k_pool)
    check("pa_decode_attention_noalloc", lib().pa_decode_attention_noalloc(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _i32(block_tables, "block_tables"),
        _i32(context_lens, "context_lens"), q.shape[0], q.shape[1], hkv, d, block_tables.shape[1],
        int(max_context_len_hint), nb, float(scale), _dtype_code(q),
        None if err_flag is None else _i32(err_flag, "err_flag"), _stream(stream)))


class BlockManager:
    """Host block manager (refcounts, block tables, copy-on-write pairs)."""

    def __init__(self, num_blocks: int):
        self._h = ctypes.c_void_p()
        check("pa_bm_create", lib().pa_bm_create(num_blocks, ctypes.byref(self._h)))
        self.num_blocks = num_blocks

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.pa_bm_destroy(h)
            self._h = None

    def add_seq(self) -> int:
        out = ctypes.c_int32()
        check("pa_bm_add_seq", lib().pa_bm_add_seq(self._h, ctypes.byref(out)))
        return out.value

    def fork(self, parent: int) -> int:
        out = ctypes.c_int32()
        check("pa_bm_fork", lib().pa_bm_fork(self._h, parent, ctypes.byref(out)))
        return out.value

    def free(self, seq: int) -> None:
        check("pa_bm_free_seq", lib().pa_bm_free_seq(self._h, seq))

    def blocks_needed(self, seq: int, start: int, n: int) -> int:
        out = ctypes.c_int32()
        check("pa_bm_blocks_needed", lib().pa_bm_blocks_needed(self._h, seq, start, n,
                                                                 ctypes.byref(out)))
        return out.value

    def prepare_append(self, seq: int, start: int, n: int) -> list:
        """Returns the copy-on-write pairs [(src, dst), ...]; raises on out-of-blocks."""
        cap = n // BLOCK_SIZE + 2
        buf = (ctypes.c_int32 * (2 * cap))()
        npairs = ctypes.c_int32()
        check("pa_bm_prepare_append", lib().pa_bm_prepare_append(
            self._h, seq, start, n, buf, cap, ctypes.byref(npairs)))
        return [(buf[2 * i], buf[2 * i + 1]) for i in range(npairs.value)]

    def truncate(self, seq: int, length: int) -> None:
        """Cuts the sequence to its first `length` tokens; the blocks behind them are let go."""
        check("pa_bm_truncate", lib().pa_bm_truncate(self._h, _bound(seq), _bound(length)))

    def block_table(self, seq: int, max_blocks: int) -> list:
        buf = (ctypes.c_int32 * max(max_blocks, 1))()
        check("pa_bm_block_table", lib().pa_bm_block_table(self._h, seq, buf, max_blocks, None))
        return list(buf[:max_blocks])

    def block_tables(self, seqs, max_blocks: int, out=None):
        """The tables of several sequences in one call: int32 array [len(seqs)][max_blocks]
        (written into `out`, a C-contiguous int32 numpy array of that shape, if given)."""
        ids = np.ascontiguousarray(np.asarray(seqs, np.int32))
        n = int(ids.size)
        if out is None:
            out = np.empty((n, max_blocks), np.int32)
        if out.dtype != np.int32 or not out.flags.c_contiguous or out.shape != (n, max_blocks):
            raise ValueError("out: a C-contiguous int32 array of shape (len(seqs), max_blocks)")
        ipp = ctypes.POINTER(ctypes.c_int32)
        check("pa_bm_block_tables", lib().pa_bm_block_tables(
            self._h, ids.ctypes.data_as(ipp), n, out.ctypes.data_as(ipp), max_blocks))
        return out

    def seq_len(self, seq: int) -> int:
        out = ctypes.c_int32()
        check("pa_bm_seq_len", lib().pa_bm_seq_len(self._h, seq, ctypes.byref(out)))
        return out.value

    def refcount(self, block: int) -> int:
        out = ctypes.c_int32()
        check("pa_bm_refcount", lib().pa_bm_refcount(self._h, block, ctypes.byref(out)))
        return out.value

    def stats(self) -> dict:
        st = BmStats()
        check("pa_bm_stats", lib().pa_bm_stats(self._h, ctypes.byref(st)))
        return {"physical_blocks": st.physical_blocks, "free_blocks": st.free_blocks,
                "logical_tokens": st.logical_tokens, "num_seqs": st.num_seqs,
                "physical_slots": st.physical_blocks * BLOCK_SIZE}
