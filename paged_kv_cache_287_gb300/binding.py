"""Thin ctypes binding of libpagedattn (the C ABI in ``include/pa.h``).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  Functions keep the C names; tensors are PyTorch CUDA tensors
whose data pointers are passed through, and the stream defaults to PyTorch's
current stream.  If the library is missing this module raises on first use:
there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpagedattn.so")

STATUS = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_CUDA",
          4: "PA_ERR_OOB", 5: "PA_ERR_TIMEOUT", 6: "PA_ERR_WORKSPACE",
          7: "PA_ERR_PRECONDITION"}

# Every symbol include/pa.h declares.
EXPORTS = ("pa_status_string", "pa_kv_block_bytes", "pa_kv_block_bytes_dtype", "pa_cache_write",
           "pa_cache_write_fp8", "pa_decode_fp8", "pa_prefill_chunk_fp8",
           "pa_decode_workspace_bytes", "pa_decode", "pa_decode_noalloc",
           "pa_decode_cascade_workspace_bytes", "pa_decode_cascade_kernels", "pa_decode_cascade",
           "pa_decode_cascade_fp8",
           "pa_prefill_chunk",
           "pa_attention_varlen_workspace_bytes", "pa_attention_varlen",
           "pa_attention_varlen_fp8", "pa_varlen_args_bytes", "pa_attention_varlen_packed",
           "pa_tree_attention_workspace_bytes", "pa_tree_attention", "pa_tree_attention_fp8",
           "pa_tree_verify", "pa_tree_accept", "pa_tree_accept_fp8", "pa_tree_attention_packed",
           "pa_tree_verify_packed", "pa_tree_accept_packed", "pa_tree_args_bytes",
           "pa_kv_block_bytes_fp4", "pa_cache_write_fp4", "pa_cache_read_fp4",
           "pa_decode_fp4_workspace_bytes", "pa_decode_fp4", "pa_qkv_rope_write",
           "pa_fp4_args_bytes",
           "pa_error_check")

# Nodes of a draft tree, at most (PA_TREE_MAX_NODES).
TREE_MAX_NODES = 64

# pa_varlen_args as laid out on a 64-bit little-endian target: out, q, k_new,
# v_new, slot_mapping, cu_q_lens, kv_cache, block_tables, seq_lens, workspace,
# workspace_bytes, stream; num_seqs, num_prefills, num_prefill_tokens,
# max_prefill_q_len, num_blocks, block_size, num_heads, num_kv_heads, head_size,
# max_blocks_per_seq, max_seq_len, kv8; scale, k_scale, v_scale.
VARLEN_ARGS = struct.Struct("<12Q12i3f")
# pa_tree_attention_args, pa_tree_verify_args and pa_tree_accept_args likewise, in the order
# of their members.
TREE_ARGS = (struct.Struct("<10Q11i3f"), struct.Struct("<11Q2q4i"), struct.Struct("<8Q8i"))
# pa_cache_fp4_args, pa_decode_fp4_args and pa_qkv_rope_write_args.
FP4_ARGS = (struct.Struct("<5Qq5i2f4x"), struct.Struct("<8Q8i3f4x"), struct.Struct("<10Qq11i3f"))
_BF16, _I32, _U8, _F32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
_tls = threading.local()  # one packed-argument buffer per thread


class PaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


_lib = None


def lib(path: Optional[str] = None):
    """Load libpagedattn.so and declare its entry points (raises if absent)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} not found: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(p)
    P, i, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_status_string.argtypes = [i]
    L.pa_kv_block_bytes.restype = sz
    L.pa_kv_block_bytes.argtypes = [i, i, i]
    L.pa_kv_block_bytes_dtype.restype = sz
    L.pa_kv_block_bytes_dtype.argtypes = [i, i, i, i]
    L.pa_cache_write_fp8.restype = i
    L.pa_cache_write_fp8.argtypes = [P, i, i, i, i, P, P, i64, P, i, ctypes.c_float,
                                     ctypes.c_float, P]
    L.pa_decode_fp8.restype = i
    L.pa_decode_fp8.argtypes = [P, P, P, i, i, i, i, i, P, i, P, i, i, ctypes.c_float,
                                ctypes.c_float, ctypes.c_float, P, sz, P]
    L.pa_prefill_chunk_fp8.restype = i
    L.pa_prefill_chunk_fp8.argtypes = [P, P, P, i, i, P, i, i, i, i, i, P, i, P, ctypes.c_float,
                                       ctypes.c_float, ctypes.c_float, P]
    L.pa_cache_write.restype = i
    L.pa_cache_write.argtypes = [P, i, i, i, i, P, P, i64, P, i, P]
    L.pa_decode_workspace_bytes.restype = sz
    L.pa_decode_workspace_bytes.argtypes = [i, i, i, i]
    L.pa_decode.restype = i
    L.pa_decode.argtypes = [P, P, P, i, i, i, i, i, P, i, P, i, i, ctypes.c_float, P, sz, P]
    L.pa_decode_noalloc.restype = i
    L.pa_decode_noalloc.argtypes = [P, P, P, i, i, i, i, i, P, i, P, i, i, ctypes.c_float, P]
    L.pa_decode_cascade_workspace_bytes.restype = sz
    L.pa_decode_cascade_workspace_bytes.argtypes = [i, i, i, i, i]
    L.pa_decode_cascade_kernels.restype = i
    L.pa_decode_cascade_kernels.argtypes = [i, i, i, i, i, i, i, i]
    L.pa_decode_cascade.restype = i
    L.pa_decode_cascade.argtypes = [P, P, P, i, i, i, i, i, P, i, P, i, i, i, ctypes.c_float, P,
                                    sz, P]
    L.pa_decode_cascade_fp8.restype = i
    L.pa_decode_cascade_fp8.argtypes = [P, P, P, i, i, i, i, i, P, i, P, i, i, i, ctypes.c_float,
                                        ctypes.c_float, ctypes.c_float, P, sz, P]
    L.pa_prefill_chunk.restype = i
    L.pa_prefill_chunk.argtypes = [P, P, P, i, i, P, i, i, i, i, i, P, i, P, ctypes.c_float, P]
    L.pa_attention_varlen_workspace_bytes.restype = sz
    L.pa_attention_varlen_workspace_bytes.argtypes = [i, i, i, i, i]
    L.pa_attention_varlen.restype = i
    L.pa_attention_varlen.argtypes = [P, P, P, P, P, P, i, i, i, i, P, i, i, i, i, i, P, i, P, i,
                                      ctypes.c_float, P, sz, P]
    L.pa_attention_varlen_fp8.restype = i
    L.pa_attention_varlen_fp8.argtypes = [P, P, P, P, P, P, i, i, i, i, P, i, i, i, i, i, P, i, P,
                                          i, ctypes.c_float, ctypes.c_float, ctypes.c_float, P,
                                          sz, P]
    L.pa_varlen_args_bytes.restype = sz
    L.pa_varlen_args_bytes.argtypes = []
    L.pa_attention_varlen_packed.restype = i
    L.pa_attention_varlen_packed.argtypes = [P]
    if L.pa_varlen_args_bytes() < VARLEN_ARGS.size:
        raise RuntimeError("pa_varlen_args is smaller than this binding's layout")
    L.pa_tree_attention_workspace_bytes.restype = sz
    L.pa_tree_attention_workspace_bytes.argtypes = [i, i, i, i, i]
    L.pa_tree_attention.restype = i
    L.pa_tree_attention.argtypes = [P, P, P, P, i, i, i, P, i, i, i, i, i, P, i, P, i,
                                    ctypes.c_float, P, sz, P]
    L.pa_tree_attention_fp8.restype = i
    L.pa_tree_attention_fp8.argtypes = [P, P, P, P, i, i, i, P, i, i, i, i, i, P, i, P, i,
                                        ctypes.c_float, ctypes.c_float, ctypes.c_float, P, sz, P]
    L.pa_tree_verify.restype = i
    L.pa_tree_verify.argtypes = [P, P, P, P, i64, P, i64, P, P, P, i, i, i, i, P, P, P]
    for f in (L.pa_tree_accept, L.pa_tree_accept_fp8):
        f.restype = i
        f.argtypes = [P, i, i, i, i, P, P, P, i, i, P, i, P, P, P]
    for f in (L.pa_tree_attention_packed, L.pa_tree_verify_packed, L.pa_tree_accept_packed):
        f.restype = i
        f.argtypes = [P]
    L.pa_tree_args_bytes.restype = sz
    L.pa_tree_args_bytes.argtypes = [i]
    for call, layout in enumerate(TREE_ARGS):
        if L.pa_tree_args_bytes(call) != layout.size:
            raise RuntimeError("the tree calls' argument structs differ from this binding's")
    L.pa_kv_block_bytes_fp4.restype = sz
    L.pa_kv_block_bytes_fp4.argtypes = [i, i, i]
    L.pa_decode_fp4_workspace_bytes.restype = sz
    L.pa_decode_fp4_workspace_bytes.argtypes = [i, i, i, i]
    for f in (L.pa_cache_write_fp4, L.pa_cache_read_fp4, L.pa_decode_fp4, L.pa_qkv_rope_write):
        f.restype = i
        f.argtypes = [P]
    L.pa_fp4_args_bytes.restype = sz
    L.pa_fp4_args_bytes.argtypes = [i]
    for call, layout in enumerate(FP4_ARGS):
        if L.pa_fp4_args_bytes(call) != layout.size:
            raise RuntimeError("the 4-bit calls' argument structs differ from this binding's")
    L.pa_error_check.restype = i
    L.pa_error_check.argtypes = [P]
    if path is None:
        _lib = L
    return L


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    try:
        return stream.cuda_stream  # torch.cuda.Stream
    except AttributeError:
        return int(stream)


def _check(status: int, where: str):
    if status != 0:
        raise PaError(status, where)


def _need(t: torch.Tensor, name: str, dtype, dims: Optional[int] = None):
    try:  # the common case in one expression (torch dtypes are singletons)
        if (t.is_cuda and t.dtype is dtype and (dims is None or t.dim() == dims)
                and t.is_contiguous() and isinstance(t, torch.Tensor)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _pool_geom(kv_cache: torch.Tensor):
    _need(kv_cache, "kv_cache", torch.bfloat16, 5)
    NB, two, Hkv, bs, D = kv_cache.shape
    if two != 2:
        raise ValueError("kv_cache must be [num_blocks, 2, num_kv_heads, block_size, head_size]")
    return NB, bs, Hkv, D


def pa_kv_block_bytes(block_size: int, num_kv_heads: int, head_size: int) -> int:
    return int(lib().pa_kv_block_bytes(block_size, num_kv_heads, head_size))


def pa_cache_write(kv_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   slot_mapping: torch.Tensor, stream=None) -> None:
    """Scatter k_new/v_new [N, Hkv, D] rows into kv_cache at slot_mapping [N]."""
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        ks = kv_cache.shape
        ok = (len(ks) == 5 and ks[1] == 2
              and kv_cache.dtype is _BF16 and kv_cache.is_cuda and kv_cache.is_contiguous()
              and k_new.dtype is _BF16 and k_new.is_cuda and k_new.is_contiguous()
              and v_new.dtype is _BF16 and v_new.is_cuda and v_new.is_contiguous()
              and slot_mapping.dtype is _I32 and slot_mapping.is_cuda
              and slot_mapping.dim() == 1 and slot_mapping.is_contiguous())
    except (AttributeError, TypeError):
        ok = False
    if not ok:
        _pool_geom(kv_cache)
        _need(k_new, "k_new", torch.bfloat16, 3)
        _need(v_new, "v_new", torch.bfloat16, 3)
        _need(slot_mapping, "slot_mapping", torch.int32, 1)
        ks = kv_cache.shape
    NB, _, Hkv, bs, D = ks
    N = slot_mapping.shape[0]
    rows = (N, Hkv, D)
    if k_new.shape != rows or v_new.shape != rows:
        raise ValueError("k_new/v_new must be [num_tokens, num_kv_heads, head_size]")
    L = _lib if _lib is not None else lib()
    _check(L.pa_cache_write(kv_cache.data_ptr(), NB, bs, Hkv, D, k_new.data_ptr(),
                            v_new.data_ptr(), Hkv * D, slot_mapping.data_ptr(), N,
                            _stream(stream)), "pa_cache_write")


def _pool8_geom(kv_cache: torch.Tensor):
    _need(kv_cache, "kv_cache", torch.uint8, 5)
    NB, two, Hkv, bs, D = kv_cache.shape
    if two != 2:
        raise ValueError("kv_cache must be [num_blocks, 2, num_kv_heads, block_size, head_size]")
    return NB, bs, Hkv, D


def pa_kv_block_bytes_dtype(block_size: int, num_kv_heads: int, head_size: int,
                            dtype_num_bytes: int) -> int:
    return int(lib().pa_kv_block_bytes_dtype(block_size, num_kv_heads, head_size,
                                             dtype_num_bytes))


def pa_cache_write_fp8(kv_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                       stream=None) -> None:
    """Quantise bf16 k_new/v_new [N, Hkv, D] into an FP8 (uint8 e4m3 codes) pool."""
    NB, bs, Hkv, D = _pool8_geom(kv_cache)
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    N = slot_mapping.shape[0]
    if k_new.shape != (N, Hkv, D) or v_new.shape != (N, Hkv, D):
        raise ValueError("k_new/v_new must be [num_tokens, num_kv_heads, head_size]")
    _check(lib().pa_cache_write_fp8(kv_cache.data_ptr(), NB, bs, Hkv, D, k_new.data_ptr(),
                                    v_new.data_ptr(), Hkv * D, slot_mapping.data_ptr(), N,
                                    float(k_scale), float(v_scale), _stream(stream)),
           "pa_cache_write_fp8")


def pa_decode_fp8(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
                  block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                  scale: float, k_scale: float, v_scale: float, workspace: torch.Tensor,
                  stream=None) -> None:
    """Decode attention over an FP8 pool (uint8 e4m3 codes times k_scale / v_scale)."""
    NB, bs, Hkv, D = _pool8_geom(kv_cache)
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(workspace, "workspace", torch.uint8, 1)
    B, Hq, Dq = q.shape
    if Dq != D or out.shape != q.shape or seq_lens.shape[0] != B or block_tables.shape[0] != B:
        raise ValueError("inconsistent decode shapes")
    _check(lib().pa_decode_fp8(out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), NB, bs, Hq,
                               Hkv, D, block_tables.data_ptr(), block_tables.shape[1],
                               seq_lens.data_ptr(), B, int(max_seq_len), float(scale),
                               float(k_scale), float(v_scale), workspace.data_ptr(),
                               workspace.numel(), _stream(stream)), "pa_decode_fp8")


def pa_prefill_chunk_fp8(out: torch.Tensor, q: torch.Tensor, cu_q_lens: torch.Tensor,
                         max_q_len: int, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                         seq_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float,
                         stream=None) -> None:
    """Chunked prefill over an FP8 pool (uint8 e4m3 codes times k_scale / v_scale)."""
    NB, bs, Hkv, D = _pool8_geom(kv_cache)
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(cu_q_lens, "cu_q_lens", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    n = seq_lens.shape[0]
    Hq = q.shape[1]
    if q.shape[2] != D or out.shape != q.shape or cu_q_lens.shape[0] != n + 1 or \
            block_tables.shape[0] != n:
        raise ValueError("inconsistent prefill shapes")
    _check(lib().pa_prefill_chunk_fp8(out.data_ptr(), q.data_ptr(), cu_q_lens.data_ptr(), n,
                                      int(max_q_len), kv_cache.data_ptr(), NB, bs, Hq, Hkv, D,
                                      block_tables.data_ptr(), block_tables.shape[1],
                                      seq_lens.data_ptr(), float(scale), float(k_scale),
                                      float(v_scale), _stream(stream)), "pa_prefill_chunk_fp8")


def pa_decode_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int,
                              head_size: int) -> int:
    return int(lib().pa_decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_size))


def pa_decode(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
              block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
              scale: float, workspace: torch.Tensor, stream=None) -> None:
    """Decode attention: q/out [B, Hq, D], block_tables [B, MB], seq_lens [B]."""
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        ks, qs, bts = kv_cache.shape, q.shape, block_tables.shape
        ok = (len(ks) == 5 and ks[1] == 2 and len(qs) == 3 and len(bts) == 2
              and kv_cache.dtype is _BF16 and kv_cache.is_cuda and kv_cache.is_contiguous()
              and q.dtype is _BF16 and q.is_cuda and q.is_contiguous()
              and out.dtype is _BF16 and out.is_cuda and out.is_contiguous()
              and block_tables.dtype is _I32 and block_tables.is_cuda
              and block_tables.is_contiguous()
              and seq_lens.dtype is _I32 and seq_lens.is_cuda and seq_lens.dim() == 1
              and seq_lens.is_contiguous()
              and workspace.dtype is _U8 and workspace.is_cuda and workspace.dim() == 1
              and workspace.is_contiguous())
    except (AttributeError, TypeError):
        ok = False
    if not ok:
        _pool_geom(kv_cache)
        _need(q, "q", torch.bfloat16, 3)
        _need(out, "out", torch.bfloat16, 3)
        _need(block_tables, "block_tables", torch.int32, 2)
        _need(seq_lens, "seq_lens", torch.int32, 1)
        _need(workspace, "workspace", torch.uint8, 1)
        ks, qs, bts = kv_cache.shape, q.shape, block_tables.shape
    NB, _, Hkv, bs, D = ks
    B, Hq, Dq = qs
    if Dq != D or out.shape != qs or seq_lens.shape[0] != B or bts[0] != B:
        raise ValueError("inconsistent decode shapes")
    L = _lib if _lib is not None else lib()
    _check(L.pa_decode(out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), NB, bs, Hq, Hkv, D,
                       block_tables.data_ptr(), bts[1], seq_lens.data_ptr(), B,
                       int(max_seq_len), float(scale), workspace.data_ptr(), workspace.numel(),
                       _stream(stream)), "pa_decode")


def pa_decode_noalloc(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                      scale: float, stream=None) -> None:
    """pa_decode with the library's built-in scratch instead of a workspace tensor."""
    NB, bs, Hkv, D = _pool_geom(kv_cache)
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, Dq = q.shape
    if Dq != D or out.shape != q.shape or seq_lens.shape[0] != B or block_tables.shape[0] != B:
        raise ValueError("inconsistent decode shapes")
    _check(lib().pa_decode_noalloc(out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), NB, bs, Hq,
                                   Hkv, D, block_tables.data_ptr(), block_tables.shape[1],
                                   seq_lens.data_ptr(), B, int(max_seq_len), float(scale),
                                   _stream(stream)), "pa_decode_noalloc")


def pa_decode_cascade_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int,
                                      head_size: int, shared_len: int) -> int:
    return int(lib().pa_decode_cascade_workspace_bytes(num_seqs, num_heads, num_kv_heads,
                                                       head_size, shared_len))


def pa_decode_cascade_kernels(num_seqs: int, num_heads: int, num_kv_heads: int, head_size: int,
                              block_size: int, max_seq_len: int, shared_len: int,
                              fp8: bool = False) -> int:
    """Kernels one pa_decode_cascade (fp8: pa_decode_cascade_fp8) call launches."""
    return int(lib().pa_decode_cascade_kernels(num_seqs, num_heads, num_kv_heads, head_size,
                                               block_size, max_seq_len, shared_len, int(fp8)))


def pa_decode_cascade(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                      shared_len: int, scale: float, workspace: torch.Tensor,
                      stream=None, kv_scales=None) -> None:
    """pa_decode for a batch whose first shared_len tokens sit in the same blocks.

    A uint8 (FP8 e4m3) pool goes to pa_decode_cascade_fp8 with
    kv_scales = (k_scale, v_scale)."""
    if kv_cache.dtype == torch.uint8:
        if kv_scales is None:
            raise ValueError("an FP8 pool needs kv_scales=(k_scale, v_scale)")
        return pa_decode_cascade_fp8(out, q, kv_cache, block_tables, seq_lens, max_seq_len,
                                     shared_len, scale, kv_scales[0], kv_scales[1], workspace,
                                     stream)
    NB, bs, Hkv, D = _pool_geom(kv_cache)
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(workspace, "workspace", torch.uint8, 1)
    B, Hq, Dq = q.shape
    if Dq != D or out.shape != q.shape or seq_lens.shape[0] != B or block_tables.shape[0] != B:
        raise ValueError("inconsistent decode shapes")
    _check(lib().pa_decode_cascade(out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), NB, bs, Hq,
                                   Hkv, D, block_tables.data_ptr(), block_tables.shape[1],
                                   seq_lens.data_ptr(), B, int(max_seq_len), int(shared_len),
                                   float(scale), workspace.data_ptr(), workspace.numel(),
                                   _stream(stream)), "pa_decode_cascade")


def pa_decode_cascade_fp8(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
                          block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                          shared_len: int, scale: float, k_scale: float, v_scale: float,
                          workspace: torch.Tensor, stream=None) -> None:
    """pa_decode_cascade over an FP8 pool (uint8 e4m3 codes times k_scale / v_scale)."""
    NB, bs, Hkv, D = _pool8_geom(kv_cache)
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(workspace, "workspace", torch.uint8, 1)
    B, Hq, Dq = q.shape
    if Dq != D or out.shape != q.shape or seq_lens.shape[0] != B or block_tables.shape[0] != B:
        raise ValueError("inconsistent decode shapes")
    _check(lib().pa_decode_cascade_fp8(out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), NB, bs,
                                       Hq, Hkv, D, block_tables.data_ptr(),
                                       block_tables.shape[1], seq_lens.data_ptr(), B,
                                       int(max_seq_len), int(shared_len), float(scale),
                                       float(k_scale), float(v_scale), workspace.data_ptr(),
                                       workspace.numel(), _stream(stream)),
           "pa_decode_cascade_fp8")


def pa_prefill_chunk(out: torch.Tensor, q: torch.Tensor, cu_q_lens: torch.Tensor,
                     max_q_len: int, kv_cache: torch.Tensor, block_tables: torch.Tensor,
                     seq_lens: torch.Tensor, scale: float, stream=None) -> None:
    """Chunked-prefill attention: q/out [sum q_len, Hq, D], cu_q_lens [n+1]."""
    NB, bs, Hkv, D = _pool_geom(kv_cache)
    _need(q, "q", torch.bfloat16, 3)
    _need(out, "out", torch.bfloat16, 3)
    _need(cu_q_lens, "cu_q_lens", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    n = seq_lens.shape[0]
    Hq = q.shape[1]
    if q.shape[2] != D or out.shape != q.shape or cu_q_lens.shape[0] != n + 1 or \
            block_tables.shape[0] != n:
        raise ValueError("inconsistent prefill shapes")
    _check(lib().pa_prefill_chunk(out.data_ptr(), q.data_ptr(), cu_q_lens.data_ptr(), n,
                                  int(max_q_len), kv_cache.data_ptr(), NB, bs, Hq, Hkv, D,
                                  block_tables.data_ptr(), block_tables.shape[1],
                                  seq_lens.data_ptr(), float(scale), _stream(stream)),
           "pa_prefill_chunk")


def pa_attention_varlen_workspace_bytes(num_seqs: int, num_prefills: int, num_heads: int,
                                        num_kv_heads: int, head_size: int) -> int:
    return int(lib().pa_attention_varlen_workspace_bytes(num_seqs, num_prefills, num_heads,
                                                         num_kv_heads, head_size))


def pa_attention_varlen(out: torch.Tensor, q: torch.Tensor, k_new: Optional[torch.Tensor],
                        v_new: Optional[torch.Tensor], slot_mapping: Optional[torch.Tensor],
                        cu_q_lens: torch.Tensor, num_prefills: int, num_prefill_tokens: int,
                        max_prefill_q_len: int, kv_cache: torch.Tensor,
                        block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                        scale: float, workspace: torch.Tensor, stream=None,
                        kv_scales: Optional[tuple] = None) -> None:
    """One step over a flattened mixed batch (chunks first, then decode tokens):
    optional cache write, chunked prefill, decode.  A uint8 kv_cache is an FP8
    (e4m3) pool and needs kv_scales = (k_scale, v_scale)."""
    fp8 = kv_cache.dtype is _U8
    if fp8 and kv_scales is None:
        raise ValueError("an FP8 pool needs kv_scales=(k_scale, v_scale)")
    # Every tensor's device, dtype, rank and contiguity in one expression (this
    # call runs once per step of a serving loop); any failure re-runs the
    # argument-by-argument checks, which name the offending tensor.
    try:
        ks, qs, bts = kv_cache.shape, q.shape, block_tables.shape
        ok = (len(ks) == 5 and ks[1] == 2 and len(qs) == 3 and len(bts) == 2
              and kv_cache.is_cuda and kv_cache.is_contiguous()
              and q.dtype is _BF16 and q.is_cuda and q.is_contiguous()
              and out.dtype is _BF16 and out.is_cuda and out.is_contiguous()
              and cu_q_lens.dtype is _I32 and cu_q_lens.is_cuda and cu_q_lens.dim() == 1
              and cu_q_lens.is_contiguous()
              and block_tables.dtype is _I32 and block_tables.is_cuda
              and block_tables.is_contiguous()
              and seq_lens.dtype is _I32 and seq_lens.is_cuda and seq_lens.dim() == 1
              and seq_lens.is_contiguous()
              and workspace.dtype is _U8 and workspace.is_cuda and workspace.dim() == 1
              and workspace.is_contiguous()
              and (fp8 or kv_cache.dtype is _BF16))
    except (AttributeError, TypeError):
        ok = False
    if not ok:
        (_pool8_geom if fp8 else _pool_geom)(kv_cache)
        _need(q, "q", torch.bfloat16, 3)
        _need(out, "out", torch.bfloat16, 3)
        _need(cu_q_lens, "cu_q_lens", torch.int32, 1)
        _need(block_tables, "block_tables", torch.int32, 2)
        _need(seq_lens, "seq_lens", torch.int32, 1)
        _need(workspace, "workspace", torch.uint8, 1)
        ks, qs, bts = kv_cache.shape, q.shape, block_tables.shape
    NB, _, Hkv, bs, D = ks
    B = seq_lens.shape[0]
    rows, Hq, Dq = qs
    if Dq != D or out.shape != qs or bts[0] != B or \
            rows != num_prefill_tokens + B - num_prefills:
        raise ValueError("inconsistent varlen shapes")
    kp = vp = sp = 0
    if slot_mapping is not None:
        try:
            ok = (k_new.dtype is _BF16 and k_new.is_cuda and k_new.is_contiguous()
                  and v_new.dtype is _BF16 and v_new.is_cuda and v_new.is_contiguous()
                  and slot_mapping.dtype is _I32 and slot_mapping.is_cuda
                  and slot_mapping.is_contiguous())
        except (AttributeError, TypeError):
            ok = False
        if not ok:
            _need(k_new, "k_new", torch.bfloat16, 3)
            _need(v_new, "v_new", torch.bfloat16, 3)
            _need(slot_mapping, "slot_mapping", torch.int32, 1)
        kv_rows = (rows, Hkv, D)
        if k_new.shape != kv_rows or v_new.shape != kv_rows or slot_mapping.shape != (rows,):
            raise ValueError("k_new/v_new [rows, num_kv_heads, head_size] and slot_mapping "
                             "[rows]: one row per query row")
        kp, vp, sp = k_new.data_ptr(), v_new.data_ptr(), slot_mapping.data_ptr()
    L = _lib if _lib is not None else lib()
    try:
        buf, addr = _tls.varlen
    except AttributeError:
        buf = ctypes.create_string_buffer(L.pa_varlen_args_bytes())
        addr = ctypes.addressof(buf)
        _tls.varlen = (buf, addr)
    if fp8:
        ks, vs = float(kv_scales[0]), float(kv_scales[1])
    else:
        ks = vs = 1.0
    # One struct and one foreign call: per-argument conversion would cost more
    # than the call itself.
    VARLEN_ARGS.pack_into(
        buf, 0, out.data_ptr(), q.data_ptr(), kp, vp, sp, cu_q_lens.data_ptr(),
        kv_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream(stream) or 0, B, int(num_prefills), int(num_prefill_tokens),
        int(max_prefill_q_len), NB, bs, Hq, Hkv, D, bts[1], int(max_seq_len), fp8,
        float(scale), ks, vs)
    st = L.pa_attention_varlen_packed(addr)
    if st:
        raise PaError(st, "pa_attention_varlen_fp8" if fp8 else "pa_attention_varlen")


def pa_tree_attention_workspace_bytes(num_seqs: int, max_tree_len: int, num_heads: int,
                                      num_kv_heads: int, head_size: int) -> int:
    return int(lib().pa_tree_attention_workspace_bytes(num_seqs, max_tree_len, num_heads,
                                                       num_kv_heads, head_size))


def _same_device(first: torch.Tensor, *others: torch.Tensor) -> None:
    for t in others:
        if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != first.get_device():
            raise ValueError("every tensor of a call must be on one device")


def _launch_stream(stream, dev: int) -> int:
    """The stream of a call whose tensors are on device dev.  The library launches on the
    current device: tensors elsewhere are refused.  (The current stream's handle is read
    without building a Stream object, which would cost more than the launch.)"""
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def _tree_args():
    """This thread's buffer for the tree calls' arguments, and its address."""
    try:
        return _tls.tree
    except AttributeError:
        buf = ctypes.create_string_buffer(max(layout.size for layout in TREE_ARGS))
        _tls.tree = (buf, ctypes.addressof(buf))
        return _tls.tree


def _tree_attention(fp8, out, q, cu_tree_lens, parents, max_tree_len, kv_cache, block_tables,
                    seq_lens, max_seq_len, scale, scales, workspace, stream):
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        dev = kv_cache.get_device()
        NB, two, Hkv, bs, D = kv_cache.shape
        rows, Hq, Dq = qs = q.shape
        B, MB = block_tables.shape
        ok = (two == 2 and Dq == D and dev >= 0
              and out.shape == qs and cu_tree_lens.shape == (B + 1,)
              and parents.shape == (rows,) and seq_lens.shape == (B,) and workspace.dim() == 1
              and kv_cache.dtype is (_U8 if fp8 else _BF16) and kv_cache.is_contiguous()
              and q.dtype is _BF16 and q.get_device() == dev and q.is_contiguous()
              and out.dtype is _BF16 and out.get_device() == dev and out.is_contiguous()
              and cu_tree_lens.dtype is _I32 and cu_tree_lens.get_device() == dev
              and cu_tree_lens.is_contiguous()
              and parents.dtype is _I32 and parents.get_device() == dev
              and parents.is_contiguous()
              and block_tables.dtype is _I32 and block_tables.get_device() == dev
              and block_tables.is_contiguous()
              and seq_lens.dtype is _I32 and seq_lens.get_device() == dev
              and seq_lens.is_contiguous()
              and workspace.dtype is _U8 and workspace.get_device() == dev
              and workspace.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        (_pool8_geom if fp8 else _pool_geom)(kv_cache)
        _need(q, "q", _BF16, 3)
        _need(out, "out", _BF16, 3)
        _need(cu_tree_lens, "cu_tree_lens", _I32, 1)
        _need(parents, "parents", _I32, 1)
        _need(block_tables, "block_tables", _I32, 2)
        _need(seq_lens, "seq_lens", _I32, 1)
        _need(workspace, "workspace", _U8, 1)
        _same_device(kv_cache, q, out, cu_tree_lens, parents, block_tables, seq_lens, workspace)
        raise ValueError("inconsistent tree attention shapes")
    L = _lib if _lib is not None else lib()
    ks, vs = scales if fp8 else (1.0, 1.0)
    buf, addr = _tree_args()
    TREE_ARGS[0].pack_into(
        buf, 0, out.data_ptr(), q.data_ptr(), cu_tree_lens.data_ptr(), parents.data_ptr(),
        kv_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _launch_stream(stream, dev) or 0, B, rows, max_tree_len, NB, bs, Hq,
        Hkv, D, MB, max_seq_len, fp8, scale, ks, vs)
    st = L.pa_tree_attention_packed(addr)
    if st:
        raise PaError(st, "pa_tree_attention_fp8" if fp8 else "pa_tree_attention")


def pa_tree_attention(out: torch.Tensor, q: torch.Tensor, cu_tree_lens: torch.Tensor,
                      parents: torch.Tensor, max_tree_len: int, kv_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                      scale: float, workspace: torch.Tensor, stream=None,
                      kv_scales: Optional[tuple] = None) -> None:
    """Attention of draft trees: q/out [total_nodes, Hq, D], parents [total_nodes],
    cu_tree_lens [B+1]; seq_lens counts context and tree.

    A uint8 (FP8 e4m3) pool goes to pa_tree_attention_fp8 with
    kv_scales = (k_scale, v_scale)."""
    fp8 = getattr(kv_cache, "dtype", None) is _U8
    if fp8 and kv_scales is None:
        raise ValueError("an FP8 pool needs kv_scales=(k_scale, v_scale)")
    _tree_attention(fp8, out, q, cu_tree_lens, parents, max_tree_len, kv_cache, block_tables,
                    seq_lens, max_seq_len, scale, kv_scales, workspace, stream)


def pa_tree_attention_fp8(out: torch.Tensor, q: torch.Tensor, cu_tree_lens: torch.Tensor,
                          parents: torch.Tensor, max_tree_len: int, kv_cache: torch.Tensor,
                          block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                          scale: float, k_scale: float, v_scale: float, workspace: torch.Tensor,
                          stream=None) -> None:
    """pa_tree_attention over an FP8 pool (uint8 e4m3 codes times k_scale / v_scale)."""
    _tree_attention(True, out, q, cu_tree_lens, parents, max_tree_len, kv_cache, block_tables,
                    seq_lens, max_seq_len, scale, (k_scale, v_scale), workspace, stream)


def _prob_rows(t: torch.Tensor, name: str, rows: int, vocab: int) -> int:
    """Row stride of a [rows, vocab] fp32 tensor whose rows may lie further apart."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not _F32:
        raise ValueError(f"{name} must be {_F32}, got {t.dtype}")
    if t.shape != (rows, vocab):
        raise ValueError(f"{name} must be [total_nodes, vocab_size]")
    s0, s1 = t.stride()
    if vocab > 1 and s1 != 1 or rows > 1 and s0 < vocab:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return s0 if rows > 1 else vocab


def pa_tree_verify(accepted: torch.Tensor, num_accepted: torch.Tensor, next_tokens: torch.Tensor,
                   target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor],
                   tokens: torch.Tensor, cu_tree_lens: torch.Tensor, parents: torch.Tensor,
                   accept_u: torch.Tensor, sample_u: torch.Tensor, stream=None) -> None:
    """Accept drafted tokens: target_probs / draft_probs [total_nodes, V] fp32 (rows may
    be strided; draft_probs None: tokens proposed without probabilities), tokens, parents,
    accept_u [total_nodes], sample_u [B]; writes accepted [B, max_tree_len] (node indices,
    -1 padded), num_accepted [B] and next_tokens [B]."""
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        dev = accepted.get_device()
        B, max_tree = accepted.shape
        rows, V = target_probs.shape
        per_seq, per_node = (B,), (rows,)
        ok = (dev >= 0 and accepted.dtype is _I32 and accepted.is_contiguous()
              and num_accepted.shape == per_seq and num_accepted.dtype is _I32
              and num_accepted.get_device() == dev and num_accepted.is_contiguous()
              and next_tokens.shape == per_seq and next_tokens.dtype is _I32
              and next_tokens.get_device() == dev and next_tokens.is_contiguous()
              and tokens.shape == per_node and tokens.dtype is _I32
              and tokens.get_device() == dev and tokens.is_contiguous()
              and cu_tree_lens.shape == (B + 1,) and cu_tree_lens.dtype is _I32
              and cu_tree_lens.get_device() == dev and cu_tree_lens.is_contiguous()
              and parents.shape == per_node and parents.dtype is _I32
              and parents.get_device() == dev and parents.is_contiguous()
              and accept_u.shape == per_node and accept_u.dtype is _F32
              and accept_u.get_device() == dev and accept_u.is_contiguous()
              and sample_u.shape == per_seq and sample_u.dtype is _F32
              and sample_u.get_device() == dev and sample_u.is_contiguous()
              and target_probs.get_device() == dev
              and (draft_probs is None or draft_probs.get_device() == dev))
        # Rows of probabilities may lie apart: the rest of _prob_rows' checks, at once.
        ts, one = target_probs.stride()
        plain = target_probs.dtype is _F32 and one == 1 and ts >= V
        dp = ds = 0
        if draft_probs is not None:
            ds, one = draft_probs.stride()
            plain = (plain and draft_probs.dtype is _F32 and one == 1 and ds >= V
                     and draft_probs.shape == (rows, V))
            dp = draft_probs.data_ptr()
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        _need(accepted, "accepted", _I32, 2)
        _need(num_accepted, "num_accepted", _I32, 1)
        _need(next_tokens, "next_tokens", _I32, 1)
        _need(tokens, "tokens", _I32, 1)
        _need(cu_tree_lens, "cu_tree_lens", _I32, 1)
        _need(parents, "parents", _I32, 1)
        _need(accept_u, "accept_u", _F32, 1)
        _need(sample_u, "sample_u", _F32, 1)
        for t, name in ((target_probs, "target_probs"), (draft_probs, "draft_probs")):
            if t is not None and (not isinstance(t, torch.Tensor) or not t.is_cuda):
                raise ValueError(f"{name} must be a CUDA tensor")
        _same_device(accepted, num_accepted, next_tokens, tokens, cu_tree_lens, parents,
                     accept_u, sample_u, target_probs, draft_probs)
        raise ValueError("inconsistent tree verification shapes")
    if not plain:
        ts = _prob_rows(target_probs, "target_probs", rows, V)
        if draft_probs is not None:
            ds = _prob_rows(draft_probs, "draft_probs", rows, V)
    L = _lib if _lib is not None else lib()
    buf, addr = _tree_args()
    TREE_ARGS[1].pack_into(
        buf, 0, accepted.data_ptr(), num_accepted.data_ptr(), next_tokens.data_ptr(),
        target_probs.data_ptr(), dp, tokens.data_ptr(), cu_tree_lens.data_ptr(),
        parents.data_ptr(), accept_u.data_ptr(), sample_u.data_ptr(),
        _launch_stream(stream, dev) or 0, ts, ds, B, rows, max_tree, V)
    st = L.pa_tree_verify_packed(addr)
    if st:
        raise PaError(st, "pa_tree_verify")


def pa_tree_accept(kv_cache: torch.Tensor, accepted: torch.Tensor, num_accepted: torch.Tensor,
                   cu_tree_lens: torch.Tensor, block_tables: torch.Tensor,
                   seq_lens: torch.Tensor, new_seq_lens: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Move the accepted nodes' K/V rows (accepted [B, max_tree_len], num_accepted [B])
    up behind their contexts, in place, in a bf16 or uint8 (FP8) pool; new_seq_lens [B],
    if given, receives the new lengths."""
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        dev = kv_cache.get_device()
        dt = kv_cache.dtype
        NB, two, Hkv, bs, D = kv_cache.shape
        B, max_tree = accepted.shape
        tB, MB = block_tables.shape
        per_seq = (B,)
        ok = (two == 2 and dev >= 0 and tB == B and (dt is _BF16 or dt is _U8)
              and kv_cache.is_contiguous()
              and accepted.dtype is _I32 and accepted.get_device() == dev
              and accepted.is_contiguous()
              and num_accepted.shape == per_seq and num_accepted.dtype is _I32
              and num_accepted.get_device() == dev and num_accepted.is_contiguous()
              and cu_tree_lens.shape == (B + 1,) and cu_tree_lens.dtype is _I32
              and cu_tree_lens.get_device() == dev and cu_tree_lens.is_contiguous()
              and block_tables.dtype is _I32 and block_tables.get_device() == dev
              and block_tables.is_contiguous()
              and seq_lens.shape == per_seq and seq_lens.dtype is _I32
              and seq_lens.get_device() == dev and seq_lens.is_contiguous()
              and (new_seq_lens is None
                   or new_seq_lens.shape == per_seq and new_seq_lens.dtype is _I32
                   and new_seq_lens.get_device() == dev and new_seq_lens.is_contiguous()))
    except (AttributeError, TypeError, ValueError):
        ok = False
    if not ok:
        (_pool8_geom if getattr(kv_cache, "dtype", None) is _U8 else _pool_geom)(kv_cache)
        _need(accepted, "accepted", _I32, 2)
        _need(num_accepted, "num_accepted", _I32, 1)
        _need(cu_tree_lens, "cu_tree_lens", _I32, 1)
        _need(block_tables, "block_tables", _I32, 2)
        _need(seq_lens, "seq_lens", _I32, 1)
        if new_seq_lens is not None:
            _need(new_seq_lens, "new_seq_lens", _I32, 1)
        _same_device(kv_cache, accepted, num_accepted, cu_tree_lens, block_tables, seq_lens,
                     new_seq_lens)
        raise ValueError("inconsistent tree acceptance shapes")
    L = _lib if _lib is not None else lib()
    buf, addr = _tree_args()
    TREE_ARGS[2].pack_into(
        buf, 0, kv_cache.data_ptr(), accepted.data_ptr(), num_accepted.data_ptr(),
        cu_tree_lens.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
        0 if new_seq_lens is None else new_seq_lens.data_ptr(), _launch_stream(stream, dev) or 0,
        NB, bs, Hkv, D, B, max_tree, MB, dt is _U8)
    st = L.pa_tree_accept_packed(addr)
    if st:
        raise PaError(st, "pa_tree_accept_fp8" if dt is _U8 else "pa_tree_accept")


def pa_kv_block_bytes_fp4(block_size: int, num_kv_heads: int, head_size: int) -> int:
    return int(lib().pa_kv_block_bytes_fp4(block_size, num_kv_heads, head_size))


def fp4_pool_shape(num_blocks: int, num_kv_heads: int, block_size: int, head_size: int) -> tuple:
    """Shape of a 4-bit pool (uint8): K's and V's tile of every (block, KV head)."""
    return num_blocks, num_kv_heads, 2, block_size * head_size * 9 // 16


def _fp4_args():
    """This thread's buffer for the 4-bit calls' arguments, and its address."""
    try:
        return _tls.fp4
    except AttributeError:
        buf = ctypes.create_string_buffer(max(layout.size for layout in FP4_ARGS))
        _tls.fp4 = (buf, ctypes.addressof(buf))
        return _tls.fp4


def _pool4_geom(kv_cache: torch.Tensor, head_size: int):
    """Blocks, block size and KV heads of a 4-bit pool of heads of head_size."""
    _need(kv_cache, "kv_cache", _U8, 4)
    NB, Hkv, two, tile = kv_cache.shape
    bs, rest = divmod(tile * 16, head_size * 9) if head_size > 0 else (0, 1)
    if two != 2 or rest:
        raise ValueError("kv_cache must be [num_blocks, num_kv_heads, 2, block_size * head_size "
                         "* 9 / 16]")
    return NB, bs, Hkv


def _head_rows(t: torch.Tensor, name: str) -> int:
    """Row stride of bf16 [rows, heads, D] whose rows may lie further apart."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [num_tokens, num_kv_heads, head_size]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if d > 1 and s2 != 1 or h > 1 and s1 != d or n > 1 and s0 < h * d:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return s0 if n > 1 else h * d


def _cache_fp4(where, k, v, kv_cache, slot_mapping, k_scale, v_scale, stream):
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        dev = kv_cache.get_device()
        NB, Hkv, two, tile = kv_cache.shape
        N, heads, D = k.shape
        bs, rest = divmod(tile * 16, D * 9)
        stride = k.stride()
        ok = (two == 2 and not rest and heads == Hkv and dev >= 0 and v.shape == k.shape
              and kv_cache.dtype is _U8 and kv_cache.is_contiguous()
              and k.dtype is _BF16 and k.get_device() == dev
              and v.dtype is _BF16 and v.get_device() == dev
              and stride == v.stride() and stride[2] == 1 and stride[1] == D
              and (stride[0] >= heads * D or N <= 1)
              and slot_mapping.shape == (N,) and slot_mapping.dtype is _I32
              and slot_mapping.get_device() == dev and slot_mapping.is_contiguous())
        stride = stride[0] if N > 1 else heads * D
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        ok = False
    if not ok:
        stride = _head_rows(k, "K rows")
        if _head_rows(v, "V rows") != stride:
            raise ValueError("K and V rows must have one row stride")
        _need(slot_mapping, "slot_mapping", _I32, 1)
        N, heads, D = k.shape
        NB, bs, Hkv = _pool4_geom(kv_cache, D)
        dev = kv_cache.get_device()
        _same_device(kv_cache, k, v, slot_mapping)
        if v.shape != k.shape or heads != Hkv or slot_mapping.shape != (N,):
            raise ValueError("K and V rows must be [num_tokens, num_kv_heads, head_size], "
                             "slot_mapping [num_tokens]")
    L = _lib if _lib is not None else lib()
    buf, addr = _fp4_args()
    FP4_ARGS[0].pack_into(buf, 0, kv_cache.data_ptr(), k.data_ptr(), v.data_ptr(),
                          slot_mapping.data_ptr(), _launch_stream(stream, dev) or 0, stride, NB,
                          bs, Hkv, D, N, k_scale, v_scale)
    st = getattr(L, where)(addr)
    if st:
        raise PaError(st, where)


def pa_cache_write_fp4(kv_cache: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                       stream=None) -> None:
    """Quantise bf16 k_new/v_new [N, Hkv, D] (rows may be strided, alike) into their slots [N] of
    a 4-bit pool (see fp4_pool_shape)."""
    _cache_fp4("pa_cache_write_fp4", k_new, v_new, kv_cache, slot_mapping, k_scale, v_scale,
               stream)


def pa_cache_read_fp4(k_out: torch.Tensor, v_out: torch.Tensor, kv_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, k_scale: float, v_scale: float,
                      stream=None) -> None:
    """The K and V rows in slots [N] of a 4-bit pool, in bf16, to k_out/v_out [N, Hkv, D] (rows
    may be strided, alike); a negative slot leaves its row as it was."""
    _cache_fp4("pa_cache_read_fp4", k_out, v_out, kv_cache, slot_mapping, k_scale, v_scale,
               stream)


def pa_decode_fp4_workspace_bytes(num_seqs: int, num_heads: int, num_kv_heads: int,
                                  head_size: int) -> int:
    return int(lib().pa_decode_fp4_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_size))


def pa_decode_fp4(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
                  block_tables: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                  scale: float, k_scale: float, v_scale: float, workspace: torch.Tensor,
                  stream=None) -> None:
    """Decode attention over a 4-bit pool: q/out [B, Hq, D], block_tables [B, MB], seq_lens
    [B]."""
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        dev = kv_cache.get_device()
        NB, Hkv, two, tile = kv_cache.shape
        B, Hq, D = qs = q.shape
        bs, rest = divmod(tile * 16, D * 9)
        tB, MB = block_tables.shape
        ok = (two == 2 and not rest and tB == B and dev >= 0
              and out.shape == qs and seq_lens.shape == (B,) and workspace.dim() == 1
              and kv_cache.dtype is _U8 and kv_cache.is_contiguous()
              and q.dtype is _BF16 and q.get_device() == dev and q.is_contiguous()
              and out.dtype is _BF16 and out.get_device() == dev and out.is_contiguous()
              and block_tables.dtype is _I32 and block_tables.get_device() == dev
              and block_tables.is_contiguous()
              and seq_lens.dtype is _I32 and seq_lens.get_device() == dev
              and seq_lens.is_contiguous()
              and workspace.dtype is _U8 and workspace.get_device() == dev
              and workspace.is_contiguous())
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        ok = False
    if not ok:
        _need(q, "q", _BF16, 3)
        _need(out, "out", _BF16, 3)
        _pool4_geom(kv_cache, q.shape[2])
        _need(block_tables, "block_tables", _I32, 2)
        _need(seq_lens, "seq_lens", _I32, 1)
        _need(workspace, "workspace", _U8, 1)
        _same_device(kv_cache, q, out, block_tables, seq_lens, workspace)
        raise ValueError("inconsistent decode shapes")
    L = _lib if _lib is not None else lib()
    buf, addr = _fp4_args()
    FP4_ARGS[1].pack_into(
        buf, 0, out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _launch_stream(stream, dev) or 0, B, NB, bs, Hq, Hkv, D, MB, max_seq_len, scale, k_scale,
        v_scale)
    st = L.pa_decode_fp4(addr)
    if st:
        raise PaError(st, "pa_decode_fp4")


def _rope_geom(q_out, kv_cache):
    """Blocks, block size, KV heads and bits per element of any pool, by its type and rank."""
    if kv_cache.dim() == 4:
        return (*_pool4_geom(kv_cache, q_out.shape[2]), 4)
    fp8 = kv_cache.dtype is _U8
    NB, bs, Hkv, D = (_pool8_geom if fp8 else _pool_geom)(kv_cache)
    if D != q_out.shape[2]:
        raise ValueError("q_out and kv_cache must have one head_size")
    return NB, bs, Hkv, 8 if fp8 else 16


def pa_qkv_rope_write(q_out: torch.Tensor, qkv: torch.Tensor, kv_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                      q_weight: Optional[torch.Tensor] = None,
                      k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      pair_axis: Optional[torch.Tensor] = None, interleaved: bool = False,
                      kv_scales: Optional[tuple] = None, stream=None) -> None:
    """Norms of q and k per head (q_weight/k_weight [D] bf16, or none), rotary positions, q to
    q_out [N, Hq, D], K and V into their slots [N] of the pool, from the projection's rows qkv
    [N, (Hq + 2 Hkv) * D] (rows may be strided).

    positions [N] or [axes, N] int32; cos_sin [positions, rot_dim] fp32 (cosines, then sines);
    pair_axis [rot_dim / 2] int32 names each pair's axis (needed for several).  The pool is bf16
    or uint8 FP8 [blocks, 2, Hkv, bs, D], or 4-bit (see fp4_pool_shape); the latter two need
    kv_scales = (k_scale, v_scale)."""
    try:  # every tensor at once; on failure the per-argument checks name the culprit
        dev = kv_cache.get_device()
        dt = kv_cache.dtype
        N, Hq, D = q_out.shape
        if kv_cache.dim() == 5:
            NB, two, Hkv, bs, rest = kv_cache.shape
            rest -= D
            bits = 16 if dt is _BF16 else 8
        else:
            NB, Hkv, two, tile = kv_cache.shape
            bs, rest = divmod(tile * 16, D * 9)
            bits = 4
        ps = positions.shape
        axes, cols = ps if len(ps) == 2 else (1, *ps)
        max_pos, rot = cos_sin.shape
        width = (Hq + 2 * Hkv) * D
        s0, s1 = qkv.stride()
        ok = (two == 2 and not rest and dev >= 0 and (dt is _U8 or bits == 16)
              and kv_cache.is_contiguous()
              and qkv.shape == (N, width) and cols == N and s1 == 1 and (s0 >= width or N <= 1)
              and q_out.dtype is _BF16 and q_out.get_device() == dev and q_out.is_contiguous()
              and qkv.dtype is _BF16 and qkv.get_device() == dev
              and slot_mapping.shape == (N,) and slot_mapping.dtype is _I32
              and slot_mapping.get_device() == dev and slot_mapping.is_contiguous()
              and positions.dtype is _I32 and positions.get_device() == dev
              and positions.is_contiguous()
              and cos_sin.dtype is _F32 and cos_sin.get_device() == dev
              and cos_sin.is_contiguous()
              and (axes == 1 or pair_axis is not None))
        qw = kw = pa = 0
        if q_weight is not None:
            ok = (ok and q_weight.shape == (D,) and q_weight.dtype is _BF16
                  and q_weight.get_device() == dev and q_weight.is_contiguous())
            qw = q_weight.data_ptr()
        if k_weight is not None:
            ok = (ok and k_weight.shape == (D,) and k_weight.dtype is _BF16
                  and k_weight.get_device() == dev and k_weight.is_contiguous())
            kw = k_weight.data_ptr()
        if pair_axis is not None:
            ok = (ok and pair_axis.shape == (rot // 2,) and pair_axis.dtype is _I32
                  and pair_axis.get_device() == dev and pair_axis.is_contiguous())
            pa = pair_axis.data_ptr()
        if N <= 1:
            s0 = width
    except (AttributeError, TypeError, ValueError, ZeroDivisionError):
        ok = False
    if not ok:
        _need(q_out, "q_out", _BF16, 3)
        if not isinstance(kv_cache, torch.Tensor):
            raise ValueError("kv_cache must be a CUDA tensor")
        _rope_geom(q_out, kv_cache)
        _need(slot_mapping, "slot_mapping", _I32, 1)
        _need(positions, "positions", _I32)
        _need(cos_sin, "cos_sin", _F32, 2)
        for t, name, dtype in ((q_weight, "q_weight", _BF16), (k_weight, "k_weight", _BF16),
                               (pair_axis, "pair_axis", _I32)):
            if t is not None:
                _need(t, name, dtype, 1)
        if not isinstance(qkv, torch.Tensor) or not qkv.is_cuda or qkv.dtype is not _BF16:
            raise ValueError(f"qkv must be a CUDA tensor of {_BF16}")
        _same_device(kv_cache, q_out, qkv, slot_mapping, positions, cos_sin, q_weight, k_weight,
                     pair_axis)
        raise ValueError("inconsistent shapes: qkv [N, (Hq + 2 Hkv) * D] of contiguous rows, "
                         "positions [N] or [axes, N] (several axes need pair_axis [rot_dim / 2]), "
                         "cos_sin [positions, rot_dim], weights [D]")
    ks, vs = kv_scales if bits != 16 and kv_scales is not None else (1.0, 1.0)
    if bits != 16 and kv_scales is None:
        raise ValueError("an FP8 or 4-bit pool needs kv_scales=(k_scale, v_scale)")
    L = _lib if _lib is not None else lib()
    buf, addr = _fp4_args()
    FP4_ARGS[2].pack_into(
        buf, 0, q_out.data_ptr(), kv_cache.data_ptr(), qkv.data_ptr(), qw, kw,
        cos_sin.data_ptr(), positions.data_ptr(), pa, slot_mapping.data_ptr(),
        _launch_stream(stream, dev) or 0, s0, N, NB, bs, Hq, Hkv, D, rot, max_pos, axes,
        bool(interleaved), bits, eps, ks, vs)
    st = L.pa_qkv_rope_write(addr)
    if st:
        raise PaError(st, "pa_qkv_rope_write")


def pa_error_check(stream=None) -> None:
    """Synchronise the stream and raise if a kernel flagged bad device data."""
    _check(lib().pa_error_check(_stream(stream)), "pa_error_check")
