"""ctypes binding of libpa_b200.so (include/pa.h).  Argument marshalling only.

Every step of the path runs in the library's CUDA kernels; PyTorch supplies
device memory and the current stream.  Loading fails loudly when the library
has not been built -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpa_b200.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libpa_b200.so is not built ({_LIB_PATH}); run "
                      "`python -m paged_kv_cache_464_b200.build`")

_lib = ctypes.CDLL(_LIB_PATH)
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

_lib.pa_reshape_and_cache.restype = _I
_lib.pa_reshape_and_cache.argtypes = [_P, _P, _P, _P, _P, _I, _I64, _I, _I, _I, _I, _P]
_lib.pa_decode_partition_size.restype = _I
_lib.pa_decode_partition_size.argtypes = [_I, _I, _I, _I, _I, _I]
_lib.pa_decode_workspace_bytes.restype = _SZ
_lib.pa_decode_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
_lib.pa_decode.restype = _I
_lib.pa_decode.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _I, _P, _SZ, _I64, _I, _I, _I, _I, _P]
_lib.pa_decode_append.restype = _I
_lib.pa_decode_append.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _I, _P, _SZ, _I64, _I, _I, _I,
                                  _I, _P]
_lib.pa_decode_static_workspace.restype = _I
_lib.pa_decode_static_workspace.argtypes = [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _I, _I64, _I, _I, _I, _I,
                                            _P]
_lib.pa_reshape_and_cache_fp8.restype = _I
_lib.pa_reshape_and_cache_fp8.argtypes = [_P, _P, _P, _P, _P, _I, _I64, _I, _I, _I, _I, _F, _F, _P]
_lib.pa_decode_fp8.restype = _I
_lib.pa_decode_fp8.argtypes = [_P, _P, _P, _P, _F, _F, _P, _I, _P, _I, _I, _I, _F, _I, _P, _SZ, _I64, _I, _I, _I, _I,
                               _P]
_lib.pa_prefill.restype = _I
_lib.pa_prefill.argtypes = [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _F, _I64, _I, _I, _I, _I, _P]
_D = ctypes.c_double
_lib.pa_rope_table.restype = _I
_lib.pa_rope_table.argtypes = [_P, _I, _I, _D, _P]
_lib.pa_rope_and_cache.restype = _I
_lib.pa_rope_and_cache.argtypes = [_P] * 9 + [_I] + [_I64] * 4 + [_I, _I, _I, _I64, _I, _I, _I, _I, _I, _P]
_lib.pa_rope_and_cache_fp8.restype = _I
_lib.pa_rope_and_cache_fp8.argtypes = [_P] * 9 + [_I] + [_I64] * 4 + [_I, _I, _I, _I64, _I, _I, _I, _I, _I, _F, _F, _P]
_lib.pa_decode_shared_prefix_workspace_bytes.restype = _SZ
_lib.pa_decode_shared_prefix_workspace_bytes.argtypes = [_I] * 8
_lib.pa_decode_shared_prefix.restype = _I
_lib.pa_decode_shared_prefix.argtypes = [_P] * 5 + [_I] + [_P] * 3 + [_I] * 6 + [_F, _P, _SZ, _I64, _I, _I, _I, _I, _P]
_lib.pa_update_block_bounds.restype = _I
_lib.pa_update_block_bounds.argtypes = [_P] * 3 + [_I] + [_P] * 2 + [_I, _I, _I64, _I, _I, _I, _I, _P]
_lib.pa_select_blocks_workspace_bytes.restype = _SZ
_lib.pa_select_blocks_workspace_bytes.argtypes = [_I] * 3
_lib.pa_select_blocks.restype = _I
_lib.pa_select_blocks.argtypes = [_P] * 4 + [_I, _P] + [_I] * 6 + [_P, _SZ, _I64, _I, _I, _I, _I, _P]
_lib.pa_decode_selected_workspace_bytes.restype = _SZ
_lib.pa_decode_selected_workspace_bytes.argtypes = [_I] * 5
_lib.pa_decode_selected.restype = _I
_lib.pa_decode_selected.argtypes = [_P] * 5 + [_I] + [_P] * 2 + [_I] * 3 + [_F, _P, _SZ, _I64, _I, _I, _I, _I, _P]
_lib.pa_copy_blocks.restype = _I
_lib.pa_copy_blocks.argtypes = [_P, _P, _P, _I, _I64, _I, _I, _I, _I, _P]
_lib.pa_stream_read.restype = _I
_lib.pa_stream_read.argtypes = [_P, _SZ, _P, _P]
_lib.pa_test_stall_next_launch.restype = _I
_lib.pa_test_stall_next_launch.argtypes = [_I, _I64]
_lib.pa_get_device_error.restype = _I
_lib.pa_get_device_error.argtypes = [_P, ctypes.POINTER(_I64), _I]
_lib.pa_status_string.restype = ctypes.c_char_p
_lib.pa_status_string.argtypes = [_I]

EXPORTED = ["pa_reshape_and_cache", "pa_decode_partition_size", "pa_decode_workspace_bytes", "pa_decode",
            "pa_decode_append", "pa_decode_static_workspace", "pa_reshape_and_cache_fp8", "pa_decode_fp8", "pa_prefill",
            "pa_rope_table", "pa_rope_and_cache", "pa_rope_and_cache_fp8", "pa_decode_shared_prefix_workspace_bytes",
            "pa_decode_shared_prefix", "pa_update_block_bounds", "pa_select_blocks_workspace_bytes",
            "pa_select_blocks", "pa_decode_selected_workspace_bytes", "pa_decode_selected",
            "pa_copy_blocks", "pa_stream_read", "pa_test_stall_next_launch", "pa_get_device_error", "pa_status_string"]
MAX_COPY_PAIRS = 65536       # PA_MAX_COPY_PAIRS in include/pa.h
STATIC_WORKSPACE_BYTES = 64 << 20   # PA_STATIC_WORKSPACE_BYTES in include/pa.h

DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
FP8 = 3                      # PA_FP8_E4M3: 1-byte caches held as torch.uint8 or torch.float8_e4m3fn
FP8_TORCH = (torch.uint8, torch.float8_e4m3fn)
DEVICE_ERRORS = {0: "ok", 1: "block id out of range", 2: "slot out of range", 3: "copy pair conflict",
                 4: "bad context length", 5: "wait timeout", 6: "V element out of range", 7: "position out of range",
                 8: "bad prefix group"}


class PaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_lib.pa_status_string(status).decode()}")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def _check(status: int, where: str) -> None:
    if status != 0:
        raise PaError(status, where)


def _stream(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream: Optional[torch.cuda.Stream]):
    """The stream that a call runs on, as the current one: for reading a length that may have been written on it a
    moment ago, and for allocating what only the call uses."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _largest(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> int:
    with _on(stream):
        return int(t.max().item()) if t.numel() else 0


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cache_args(k_cache: torch.Tensor, v_cache: torch.Tensor):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, num_kv_heads, head_dim]")
    if k_cache.dtype not in DTYPE_CODE and k_cache.dtype not in FP8_TORCH:
        raise ValueError(f"unsupported cache dtype {k_cache.dtype}")
    nb, bs, hkv, d = k_cache.shape
    return nb, bs, hkv, d, (FP8 if k_cache.dtype in FP8_TORCH else DTYPE_CODE[k_cache.dtype])


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write key/value rows [T, Hkv, D] into the caches at ``slot_mapping`` [T] (int64)."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    if key.dtype != k_cache.dtype or value.dtype != k_cache.dtype or slot_mapping.dtype != torch.int64:
        raise ValueError("key/value must have the cache dtype and slot_mapping must be int64")
    T = key.shape[0]
    if tuple(key.shape) != (T, hkv, d) or tuple(value.shape) != (T, hkv, d) or slot_mapping.numel() != T:
        raise ValueError("key/value must be [T, num_kv_heads, head_dim] with T slots")
    _check(_lib.pa_reshape_and_cache(_dev(key, "key"), _dev(value, "value"), _dev(k_cache, "k_cache"),
                                     _dev(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping") if T else None,
                                     T, nb, bs, hkv, d, dt, _stream(stream)), "pa_reshape_and_cache")


def decode_partition_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                          max_context_len: int, partition_size: int = 0) -> int:
    return int(_lib.pa_decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len,
                                             partition_size))


def decode_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                           max_context_len: int, partition_size: int = 0) -> int:
    return int(_lib.pa_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len,
                                              partition_size))


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
           context_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None, *,
           max_context_len: Optional[int] = None, partition_size: int = 0,
           workspace: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode attention.  q [S, Hq, D]; block_tables [S, MBS] int32; context_lens [S] int32.

    ``max_context_len`` should be passed by callers that know it (reading it
    from ``context_lens`` costs a device-to-host sync).  ``workspace`` and
    ``out`` are allocated here, on ``stream``, when needed and not given.
    """
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    S, hq, dq = q.shape
    if dq != d or q.dtype != k_cache.dtype:
        raise ValueError("q must be [S, num_heads, head_dim] with the cache dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables must be [S, max_blocks_per_seq] and context_lens [S]")
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    if max_context_len is None:
        max_context_len = _largest(context_lens, stream)
    need = decode_workspace_bytes(S, hq, hkv, d, max_context_len, partition_size)
    if need and workspace is None:
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.pa_decode(_dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                          _dev(block_tables, "block_tables"), block_tables.shape[1],
                          _dev(context_lens, "context_lens"), S, hq, max_context_len, float(scale),
                          partition_size, ws_ptr, ws_bytes, nb, bs, hkv, d, dt, _stream(stream)), "pa_decode")
    return out


def decode_append(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                  v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                  out: Optional[torch.Tensor] = None, *, max_context_len: Optional[int] = None,
                  partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Write each sequence's new token (key/value [S, Hkv, D]) at position
    context_len - 1 through its block table, then decode -- one launch."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    S, hq, dq = q.shape
    if dq != d or q.dtype != k_cache.dtype or key.dtype != k_cache.dtype or value.dtype != k_cache.dtype:
        raise ValueError("q, key and value must have the cache dtype and head_dim")
    if tuple(key.shape) != (S, hkv, d) or tuple(value.shape) != (S, hkv, d):
        raise ValueError("key/value must be [S, num_kv_heads, head_dim]")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables must be [S, max_blocks_per_seq] and context_lens [S]")
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    if max_context_len is None:
        max_context_len = _largest(context_lens, stream)
    need = decode_workspace_bytes(S, hq, hkv, d, max_context_len, partition_size)
    if need and workspace is None:
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.pa_decode_append(_dev(out, "out"), _dev(q, "q"), _dev(key, "key"), _dev(value, "value"),
                                 _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                                 _dev(block_tables, "block_tables"), block_tables.shape[1],
                                 _dev(context_lens, "context_lens"), S, hq, max_context_len, float(scale),
                                 partition_size, ws_ptr, ws_bytes, nb, bs, hkv, d, dt, _stream(stream)),
           "pa_decode_append")
    return out


def decode_static_workspace(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                            out: Optional[torch.Tensor] = None, *, max_context_len: int,
                            partition_size: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``decode`` for callers that cannot allocate device memory: the split-K
    scratch is the library's own fixed array (STATIC_WORKSPACE_BYTES per GPU),
    so the library allocates nothing.  ``out`` must be given by such callers
    (it is allocated here only as a convenience when omitted).  Calls that
    overlap on the GPU share the array and race.  Every call that needs scratch
    looks up the array's address on the current device (the first lookup may
    load the library's device code there, so make the first call on each
    device before any stream capture)."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    S, hq, dq = q.shape
    if dq != d or q.dtype != k_cache.dtype:
        raise ValueError("q must be [S, num_heads, head_dim] with the cache dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables must be [S, max_blocks_per_seq] and context_lens [S]")
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    _check(_lib.pa_decode_static_workspace(
        _dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables"), block_tables.shape[1], _dev(context_lens, "context_lens"), S, hq,
        max_context_len, float(scale), partition_size, nb, bs, hkv, d, dt, _stream(stream)),
        "pa_decode_static_workspace")
    return out


def reshape_and_cache_fp8(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                          slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                          stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise key/value rows [T, Hkv, 128] (fp16/bf16) into 1-byte E4M3 caches at their slots."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    if dt != FP8 or key.dtype not in (torch.float16, torch.bfloat16) or value.dtype != key.dtype:
        raise ValueError("1-byte caches and fp16/bf16 key/value expected")
    T = key.shape[0]
    if tuple(key.shape) != (T, hkv, d) or tuple(value.shape) != (T, hkv, d) or slot_mapping.numel() != T:
        raise ValueError("key/value must be [T, num_kv_heads, head_dim] with T slots")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    _check(_lib.pa_reshape_and_cache_fp8(_dev(key, "key"), _dev(value, "value"), _dev(k_cache, "k_cache"),
                                         _dev(v_cache, "v_cache"),
                                         _dev(slot_mapping, "slot_mapping") if T else None, T, nb, bs, hkv, d,
                                         DTYPE_CODE[key.dtype], float(k_scale), float(v_scale), _stream(stream)),
           "pa_reshape_and_cache_fp8")


def decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float, v_scale: float,
               block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
               out: Optional[torch.Tensor] = None, *, max_context_len: Optional[int] = None,
               partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode over 1-byte E4M3 caches; q/out fp16 or bf16."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    S, hq, dq = q.shape
    if dt != FP8 or q.dtype not in (torch.float16, torch.bfloat16) or dq != d:
        raise ValueError("1-byte caches and fp16/bf16 q [S, Hq, head_dim] expected")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables must be [S, max_blocks_per_seq] and context_lens [S]")
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    if max_context_len is None:
        max_context_len = _largest(context_lens, stream)
    need = decode_workspace_bytes(S, hq, hkv, d, max_context_len, partition_size)
    if need and workspace is None:
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _dev(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.pa_decode_fp8(_dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                              float(k_scale), float(v_scale), _dev(block_tables, "block_tables"),
                              block_tables.shape[1], _dev(context_lens, "context_lens"), S, hq, max_context_len,
                              float(scale), partition_size, ws_ptr, ws_bytes, nb, bs, hkv, d, DTYPE_CODE[q.dtype],
                              _stream(stream)), "pa_decode_fp8")
    return out


def prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
            context_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
            out: Optional[torch.Tensor] = None, *, max_query_len: Optional[int] = None,
            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged chunked-prefill attention.  q [T, Hq, 128]; sequence b's chunk is rows
    query_start_loc[b]:query_start_loc[b+1] (int32 [S+1]), the last tokens of its
    context_lens[b] cached tokens.  ``max_query_len`` (the longest chunk) should be
    passed by callers that know it; reading it here costs a device-to-host sync."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    T, hq, dq = q.shape
    if dq != d or q.dtype != k_cache.dtype:
        raise ValueError("q must be [T, num_heads, head_dim] with the cache dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32 or query_start_loc.dtype != torch.int32:
        raise ValueError("block_tables, context_lens and query_start_loc must be int32")
    S = context_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != S or query_start_loc.numel() != S + 1:
        raise ValueError("block_tables must be [S, MBS] and query_start_loc [S + 1]")
    if max_query_len is None:
        with _on(stream):
            qsl = query_start_loc.cpu()
        max_query_len = int((qsl[1:] - qsl[:-1]).max()) if S else 0
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must match q")
    _check(_lib.pa_prefill(_dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                           _dev(block_tables, "block_tables"), block_tables.shape[1],
                           _dev(context_lens, "context_lens"), _dev(query_start_loc, "query_start_loc"), S, hq,
                           int(max_query_len), float(scale), nb, bs, hkv, d, dt, _stream(stream)), "pa_prefill")
    return out


# -- rotate and append, shared-prefix decode, block-sparse decode
# These wrappers run on the tensors' device (which need not be the current one)
# and allocate what the caller left out on the stream that the call runs on.

# They are called once a layer and step, so the checks are a single pass and the
# messages are put together only when one fails.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _refuse(names: str, tensors, flat: int) -> None:
    """Say which of the tensors is not where the first one is, or (the first `flat` of them) not contiguous."""
    for i, (name, t) in enumerate(zip(names.split(), tensors)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != tensors[0].get_device():
            raise ValueError(f"{name} is on {t.device}, {names.split()[0]} on {tensors[0].device}")
        if i < flat and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _launch(fn, where: str, index: int, stream: Optional[torch.cuda.Stream], *args) -> None:
    if stream is None:
        raw = _raw_stream(index)
    elif stream.device_index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    else:
        raw = stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != 0:
        raise PaError(status, where)


def _empty(shape, dtype: torch.dtype, index: int, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=index)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=index)


def _bytes_of(fn, index: int, *args: int) -> int:
    """A workspace size, which may depend on the device's SM count."""
    if index == torch.cuda.current_device():
        return int(fn(*args))
    with torch.cuda.device(index):
        return int(fn(*args))


def _workspace(need: int, workspace: Optional[torch.Tensor], index: int, stream: Optional[torch.cuda.Stream]):
    """(tensor, pointer, bytes); the tensor has to live until the launch is queued."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _empty(need, torch.uint8, index, stream)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the other tensors' device")
    return workspace, workspace.data_ptr(), workspace.nbytes


def rope_table(max_position: int, rotary_dim: int, base: float = 10000.0,
               device: Optional[torch.device] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """[max_position, rotary_dim] float32: cosines, then sines, of position * base^(-2i / rotary_dim)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    table = _empty((max(max_position, 0), max(rotary_dim, 0)), torch.float32, device.index, stream)
    _launch(_lib.pa_rope_table, "pa_rope_table", device.index, stream, table.data_ptr(), max_position, rotary_dim, float(base))
    return table


def _row_stride(t: torch.Tensor, name: str, T: int, h: int, d: int) -> int:
    """Elements between the token rows of [T, h, d]; heads and d must be contiguous."""
    if T == 0:
        return h * d
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return s0 if T > 1 else h * d


def _rope(fn, where, q, key, value, positions, cos_sin, k_cache, v_cache, slot_mapping, q_out, interleaved, stream,
          dtype_code, *scales):
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, num_kv_heads, head_dim]")
    nb, bs, hkv, d = k_cache.shape
    if q.dim() != 3 or key.shape != value.shape or key.dim() != 3:
        raise ValueError("q must be [T, num_heads, head_dim], key and value [T, num_kv_heads, head_dim]")
    T, hq, dq = q.shape
    dtype = q.dtype
    if dq != d or key.shape != (T, hkv, d) or key.dtype != dtype or value.dtype != dtype:
        raise ValueError("q [T, num_heads, head_dim], key and value [T, num_kv_heads, head_dim] must have one dtype")
    if positions.dtype != torch.int64 or slot_mapping.dtype != torch.int64 or positions.numel() != T or \
            slot_mapping.numel() != T:
        raise ValueError("positions and slot_mapping must be int64 [T]")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_position, rotary_dim] float32")
    index = k_cache.get_device()
    if not (0 <= index == v_cache.get_device() == positions.get_device() == cos_sin.get_device()
            == slot_mapping.get_device() == q.get_device() == key.get_device() == value.get_device()
            and k_cache.is_contiguous() and v_cache.is_contiguous() and positions.is_contiguous()
            and cos_sin.is_contiguous() and slot_mapping.is_contiguous()):
        _refuse("k_cache v_cache positions cos_sin slot_mapping q key value",
                (k_cache, v_cache, positions, cos_sin, slot_mapping, q, key, value), 5)
    if q_out is None:
        q_out = _empty((T, hq, d), dtype, index, stream)
    elif q_out.shape != q.shape or q_out.dtype != dtype or q_out.get_device() != index:
        raise ValueError("q_out must match q")
    max_position, rotary = cos_sin.shape
    _launch(fn, where, index, stream, q_out.data_ptr(), q.data_ptr(), key.data_ptr(), value.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), slot_mapping.data_ptr(), T,
            _row_stride(q_out, "q_out", T, hq, d), _row_stride(q, "q", T, hq, d), _row_stride(key, "key", T, hkv, d),
            _row_stride(value, "value", T, hkv, d), max_position, rotary, 1 if interleaved else 0, nb, bs, hq, hkv, d,
            dtype_code, *scales)
    return q_out


def rope_and_cache(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                   cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                   q_out: Optional[torch.Tensor] = None, *, interleaved: bool = False,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Rotate q [T, Hq, D] into ``q_out`` (q itself: in place) and key [T, Hkv, D] into the cache by ``positions`` [T]
    (int64; < 0 = padding, nothing done), and write value, at ``slot_mapping`` [T] (int64; < 0 = no cache write).
    q, key, value and q_out may be slices of wider rows.  ``cos_sin``: ``rope_table``'s."""
    if k_cache.dtype not in DTYPE_CODE or q.dtype != k_cache.dtype:
        raise ValueError("q, key and value must have the cache dtype")
    return _rope(_lib.pa_rope_and_cache, "pa_rope_and_cache", q, key, value, positions, cos_sin, k_cache, v_cache,
                 slot_mapping, q_out, interleaved, stream, DTYPE_CODE[q.dtype])


def rope_and_cache_fp8(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                       cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                       q_out: Optional[torch.Tensor] = None, *, interleaved: bool = False,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``rope_and_cache`` from fp16/bf16 rows into 1-byte E4M3 caches."""
    if k_cache.dtype not in FP8_TORCH or q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("1-byte caches and fp16/bf16 q, key and value expected")
    return _rope(_lib.pa_rope_and_cache_fp8, "pa_rope_and_cache_fp8", q, key, value, positions, cos_sin, k_cache,
                 v_cache, slot_mapping, q_out, interleaved, stream, DTYPE_CODE[q.dtype], float(k_scale), float(v_scale))


def _decode_inputs(q, block_tables, context_lens, d: int, dtype: torch.dtype):
    S, hq, dq = q.shape
    if dq != d or q.dtype != dtype:
        raise ValueError("q must be [S, num_heads, head_dim] with the cache dtype")
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32:
        raise ValueError("block_tables and context_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or context_lens.numel() != S:
        raise ValueError("block_tables must be [S, max_blocks_per_seq] and context_lens [S]")
    return S, hq


def _out_like(q, out, index, stream):
    if out is None:
        return _empty(q.shape, q.dtype, index, stream)
    if out.shape != q.shape or out.dtype != q.dtype or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must match q and be contiguous")
    return out


def decode_shared_prefix_workspace_bytes(num_seqs: int, num_groups: int, num_heads: int, num_kv_heads: int,
                                         head_dim: int, max_prefix_len: int, max_suffix_len: int,
                                         max_group_size: int) -> int:
    return int(_lib.pa_decode_shared_prefix_workspace_bytes(num_seqs, num_groups, num_heads, num_kv_heads, head_dim,
                                                            max_prefix_len, max_suffix_len, max_group_size))


def decode_shared_prefix(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, group_start: torch.Tensor, prefix_lens: torch.Tensor,
                         scale: float, out: Optional[torch.Tensor] = None, *, max_prefix_len: Optional[int] = None,
                         max_suffix_len: Optional[int] = None, max_group_size: Optional[int] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode for groups of sequences with common prefixes.  Sequences group_start[i]:group_start[i+1]
    (int32 [G + 1]) share their first prefix_lens[i] (int32 [G], multiples of 16) tokens; context_lens are whole
    lengths.  Callers that know the three maxima should pass them (reading them costs a device-to-host sync)."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    S, hq = _decode_inputs(q, block_tables, context_lens, d, k_cache.dtype)
    n = prefix_lens.numel()
    if group_start.dtype != torch.int32 or prefix_lens.dtype != torch.int32 or group_start.numel() != n + 1:
        raise ValueError("group_start and prefix_lens must be int32 [G + 1] and [G]")
    index = q.get_device()
    if not (0 <= index == k_cache.get_device() == v_cache.get_device() == block_tables.get_device()
            == context_lens.get_device() == group_start.get_device() == prefix_lens.get_device()
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous() and group_start.is_contiguous()
            and prefix_lens.is_contiguous()):
        _refuse("q k_cache v_cache block_tables context_lens group_start prefix_lens",
                (q, k_cache, v_cache, block_tables, context_lens, group_start, prefix_lens), 7)
    if max_prefix_len is None or max_suffix_len is None or max_group_size is None:
        with _on(stream):
            starts, prefixes = group_start.cpu().long(), prefix_lens.cpu().long()
        sizes = (starts[1:] - starts[:-1]).clamp(min=0)
        if max_group_size is None:
            max_group_size = int(sizes.max()) if n else 0
        if max_prefix_len is None:
            max_prefix_len = int(prefixes.max()) if n else 0
        if max_suffix_len is None:
            with _on(stream):
                own = context_lens.cpu().long()
            if int(sizes.sum()) == S:
                own = own - prefixes.repeat_interleave(sizes)
            max_suffix_len = max(0, int(own.max())) if S else 0
    out = _out_like(q, out, index, stream)
    need = 0
    if workspace is None:
        need = _bytes_of(_lib.pa_decode_shared_prefix_workspace_bytes, index, S, n, hq, hkv, d, max_prefix_len,
                         max_suffix_len, max_group_size)
    workspace, ws_ptr, ws_bytes = _workspace(need, workspace, index, stream)
    _launch(_lib.pa_decode_shared_prefix, "pa_decode_shared_prefix", index, stream, out.data_ptr(), q.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
            context_lens.data_ptr(), group_start.data_ptr(), prefix_lens.data_ptr(), S, n, hq, max_prefix_len,
            max_suffix_len, max_group_size, float(scale), ws_ptr, ws_bytes, nb, bs, hkv, d, dt)
    return out


def update_block_bounds(k_cache: torch.Tensor, block_bounds: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, new_lens: torch.Tensor, *, max_new_len: Optional[int] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """Smallest and largest key per channel, ``block_bounds`` [NB, 2, Hkv, D], of every block that holds one of a
    sequence's last ``new_lens`` (int32 [S]) tokens."""
    if k_cache.dim() != 4 or k_cache.dtype not in DTYPE_CODE:
        raise ValueError("k_cache must be [num_blocks, block_size, num_kv_heads, head_dim], fp32, fp16 or bf16")
    nb, bs, hkv, d = k_cache.shape
    dt = DTYPE_CODE[k_cache.dtype]
    if block_bounds.shape != (nb, 2, hkv, d) or block_bounds.dtype != k_cache.dtype:
        raise ValueError("block_bounds must be [num_blocks, 2, num_kv_heads, head_dim] with the cache dtype")
    S = context_lens.numel()
    if block_tables.dtype != torch.int32 or context_lens.dtype != torch.int32 or new_lens.dtype != torch.int32:
        raise ValueError("block_tables, context_lens and new_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] != S or new_lens.numel() != S:
        raise ValueError("block_tables must be [S, max_blocks_per_seq], context_lens and new_lens [S]")
    index = k_cache.get_device()
    if not (0 <= index == block_bounds.get_device() == block_tables.get_device() == context_lens.get_device()
            == new_lens.get_device() and k_cache.is_contiguous() and block_bounds.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous() and new_lens.is_contiguous()):
        _refuse("k_cache block_bounds block_tables context_lens new_lens",
                (k_cache, block_bounds, block_tables, context_lens, new_lens), 5)
    if max_new_len is None:
        max_new_len = _largest(new_lens, stream)
    _launch(_lib.pa_update_block_bounds, "pa_update_block_bounds", index, stream, k_cache.data_ptr(),
            block_bounds.data_ptr(), block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(),
            new_lens.data_ptr(), S, max_new_len, nb, bs, hkv, d, dt)


def select_blocks_workspace_bytes(num_seqs: int, num_kv_heads: int, max_context_len: int) -> int:
    return int(_lib.pa_select_blocks_workspace_bytes(num_seqs, num_kv_heads, max_context_len))


def select_blocks(q: torch.Tensor, block_bounds: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, selected, *, sink_blocks: int = 1, recent_blocks: int = 1,
                  max_context_len: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The blocks each (sequence, KV head) attends to, by the score of ``block_bounds``: ``selected`` is the int32
    [S, Hkv, K] tensor to write, or K.  Ascending logical indices, -1 behind them."""
    if block_bounds.dim() != 4 or block_bounds.shape[1] != 2 or block_bounds.dtype not in DTYPE_CODE:
        raise ValueError("block_bounds must be [num_blocks, 2, num_kv_heads, head_dim]")
    nb, _, hkv, d = block_bounds.shape
    S, hq = _decode_inputs(q, block_tables, context_lens, d, block_bounds.dtype)
    index = q.get_device()
    if not (0 <= index == block_bounds.get_device() == block_tables.get_device() == context_lens.get_device()
            and q.is_contiguous() and block_bounds.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous()):
        _refuse("q block_bounds block_tables context_lens", (q, block_bounds, block_tables, context_lens), 4)
    if isinstance(selected, int):
        selected = _empty((S, hkv, max(selected, 0)), torch.int32, index, stream)
    elif selected.dtype != torch.int32 or selected.dim() != 3 or selected.shape[:2] != (S, hkv) or \
            selected.get_device() != index or not selected.is_contiguous():
        raise ValueError("selected must be a contiguous int32 [S, num_kv_heads, K]")
    if max_context_len is None:
        max_context_len = _largest(context_lens, stream)
    need = _lib.pa_select_blocks_workspace_bytes(S, hkv, max_context_len) if workspace is None else 0
    workspace, ws_ptr, ws_bytes = _workspace(need, workspace, index, stream)
    _launch(_lib.pa_select_blocks, "pa_select_blocks", index, stream, selected.data_ptr(), q.data_ptr(),
            block_bounds.data_ptr(), block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), S, hq,
            max_context_len, selected.shape[2], sink_blocks, recent_blocks, ws_ptr, ws_bytes, nb, 16, hkv, d,
            DTYPE_CODE[q.dtype])
    return selected


def decode_selected_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                    num_selected: int) -> int:
    return int(_lib.pa_decode_selected_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, num_selected))


def decode_selected(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                    context_lens: torch.Tensor, selected: torch.Tensor, scale: float,
                    out: Optional[torch.Tensor] = None, *, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Paged decode over the blocks of ``selected`` (int32 [S, Hkv, K] distinct logical indices, < 0 = none) only."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    S, hq = _decode_inputs(q, block_tables, context_lens, d, k_cache.dtype)
    if selected.dtype != torch.int32 or selected.dim() != 3 or selected.shape[:2] != (S, hkv):
        raise ValueError("selected must be int32 [S, num_kv_heads, K]")
    K = selected.shape[2]
    index = q.get_device()
    if not (0 <= index == k_cache.get_device() == v_cache.get_device() == block_tables.get_device()
            == context_lens.get_device() == selected.get_device() and q.is_contiguous() and k_cache.is_contiguous()
            and v_cache.is_contiguous() and block_tables.is_contiguous() and context_lens.is_contiguous()
            and selected.is_contiguous()):
        _refuse("q k_cache v_cache block_tables context_lens selected",
                (q, k_cache, v_cache, block_tables, context_lens, selected), 6)
    out = _out_like(q, out, index, stream)
    need = 0
    if workspace is None:
        need = _bytes_of(_lib.pa_decode_selected_workspace_bytes, index, S, hq, hkv, d, K)
    workspace, ws_ptr, ws_bytes = _workspace(need, workspace, index, stream)
    _launch(_lib.pa_decode_selected, "pa_decode_selected", index, stream, out.data_ptr(), q.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
            context_lens.data_ptr(), selected.data_ptr(), S, hq, K, float(scale), ws_ptr, ws_bytes, nb, bs, hkv, d, dt)
    return out


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_mapping: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy whole blocks (src, dst) = block_mapping[i] ([P, 2] int64) in both caches."""
    nb, bs, hkv, d, dt = _cache_args(k_cache, v_cache)
    if block_mapping.dtype != torch.int64 or (block_mapping.numel() and block_mapping.shape[-1] != 2):
        raise ValueError("block_mapping must be [P, 2] int64")
    P = block_mapping.numel() // 2
    _check(_lib.pa_copy_blocks(_dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
                               _dev(block_mapping, "block_mapping") if P else None, P, nb, bs, hkv, d, dt,
                               _stream(stream)), "pa_copy_blocks")


def stream_read(buf: torch.Tensor, sink: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Read every byte of ``buf`` once (a plain streaming read, for measuring the
    read-only bandwidth); XORs its 8-byte words into ``sink`` (one int64 on the device)."""
    if sink.dtype != torch.int64 or sink.numel() != 1:
        raise ValueError("sink must be one int64")
    _check(_lib.pa_stream_read(_dev(buf, "buf"), buf.numel() * buf.element_size(), _dev(sink, "sink"),
                               _stream(stream)), "pa_stream_read")


def test_stall_next_launch(kernel: str, cta: int) -> None:
    """Test hook: the next launch of ``kernel`` ("decode" or "prefill") leaves
    one copy of CTA ``cta`` unissued, so that CTA's bounded wait runs out
    (PA_DEV_WAIT_TIMEOUT, detail = cta) within about a millisecond; ``cta=-1``
    disarms.  "shared_prefix": the prefix kernel of ``decode_shared_prefix``."""
    _check(_lib.pa_test_stall_next_launch({"decode": 0, "prefill": 1, "shared_prefix": 3}[kernel], int(cta)),
           "pa_test_stall_next_launch")


def get_device_error(clear: bool = True, stream: Optional[torch.cuda.Stream] = None):
    """(kind, detail) of the first problem a kernel recorded on the current device."""
    detail = _I64(0)
    code = _lib.pa_get_device_error(_stream(stream), ctypes.byref(detail), 1 if clear else 0)
    if code < 0:
        raise PaError(5, "pa_get_device_error")
    return code, int(detail.value)


# -- raw entry points for callers that manage pointers themselves -----------------
raw = _lib
