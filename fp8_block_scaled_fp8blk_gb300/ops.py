"""Thin ctypes binding of libfp8blk (C ABI in ``include/fp8blk.h``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of the library.  Tensors are torch CUDA tensors (torch is used for
device memory and streams); each call enqueues on the current torch stream of
the tensors' device and returns without synchronizing.  Importing this module
loads the library and raises ``ImportError`` if it has not been built, so the
product path can never run without its kernels.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import numpy as np
import torch

from .build import LIB as _LIB_PATH

library_path = _LIB_PATH

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"libfp8blk is not built ({_LIB_PATH} missing); run "
        "`python -m fp8_block_scaled_fp8blk_gb300.build` (or __graft_entry__.build())")

_lib = ctypes.CDLL(_LIB_PATH)

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int

_lib.fp8blk_abi_version.restype = _INT
_lib.fp8blk_strerror.restype = ctypes.c_char_p
_lib.fp8blk_strerror.argtypes = [_INT]
_lib.fp8blk_scales_from_e8m0.restype = _INT
_lib.fp8blk_scales_from_e8m0.argtypes = [_P, ctypes.c_size_t, _P, ctypes.POINTER(ctypes.c_size_t)]
_lib.fp8blk_gemv.restype = _INT
_lib.fp8blk_gemv.argtypes = [_P, _P, _P, _P, _INT, _I64, _I64, _P]
_lib.fp8blk_gemv_argmax_ws_bytes.restype = ctypes.c_size_t
_lib.fp8blk_gemv_argmax_ws_bytes.argtypes = [_INT, _I64, _I64]
_lib.fp8blk_gemv_argmax.restype = _INT
_lib.fp8blk_gemv_argmax.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _INT, _I64, _I64, _P]
_lib.fp8blk_gemv_argmax_noalloc.restype = _INT
_lib.fp8blk_gemv_argmax_noalloc.argtypes = [_P, _P, _P, _P, _P, _INT, _I64, _I64, _P]
_lib.fp8blk_noalloc_scratch_bytes.restype = ctypes.c_size_t
_lib.fp8blk_bf16_gemv.restype = _INT
_lib.fp8blk_bf16_gemv.argtypes = [_P, _P, _P, _INT, _I64, _I64, _P]
_lib.nvfp4_expert_dequant.restype = _INT
_lib.nvfp4_expert_dequant.argtypes = [_P, _P, _P, _INT, _INT, _P, _I64, _I64, _P]
_lib.nvfp4_expert_dequant_gemv.restype = _INT
_lib.nvfp4_expert_dequant_gemv.argtypes = [_P, _P, _P, _INT, _P, _INT, _P, _P, _P, _I64, _I64, _P]
_lib.nvfp4_expert_gemv.restype = _INT
_lib.nvfp4_expert_gemv.argtypes = [_P, _P, _P, _INT, _P, _INT, _P, _P, _I64, _I64, _P]
_lib.mxfp4_expert_gemv.restype = _INT
_lib.mxfp4_expert_gemv.argtypes = [_P, _P, _INT, _P, _INT, _P, _P, _I64, _I64, _P]
_lib.fp8blk_kv_map.restype = _INT
_lib.fp8blk_kv_map.argtypes = [_P] * 10 + [_INT] * 4 + [_I64, _P]
_lib.fp8blk_kv_map_held.restype = _INT
_lib.fp8blk_kv_map_held.argtypes = [_P] * 12 + [_INT] * 4 + [_I64, _P]
_lib.fp8blk_kv_append.restype = _INT
_lib.fp8blk_kv_append.argtypes = [_P, _P, _INT, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _INT, _INT, _INT, _P]
_lib.fp8blk_kv_attn_ws_bytes.restype = ctypes.c_size_t
_lib.fp8blk_kv_attn_ws_bytes.argtypes = [_INT] * 5
_lib.fp8blk_kv_attn.restype = _INT
_lib.fp8blk_kv_attn.argtypes = [_P, _INT] + [_P] * 10 + [ctypes.c_size_t, _INT, _INT, _I64, _INT, _INT, _INT, _INT, _I64,
                                                       _INT, _I64, _I64, ctypes.c_float, _P]
_lib.fp8blk_token_logprobs.restype = _INT
_lib.fp8blk_token_logprobs.argtypes = [_P, _INT] + [_P] * 6 + [_I64, _I64, _I64, _INT, _P]
_lib.fp8blk_set_launch_tuning.restype = _INT
_lib.fp8blk_set_launch_tuning.argtypes = [_INT, _INT, _INT, _INT, _INT]
_lib.fp8blk_set_m1_kernel.restype = _INT
_lib.fp8blk_set_m1_kernel.argtypes = [_INT, _I64]
_lib.fp8blk_set_fp4_kernel.restype = _INT
_lib.fp8blk_set_fp4_kernel.argtypes = [_INT]
_lib.fp8blk_set_wait_limit.restype = _INT
_lib.fp8blk_set_wait_limit.argtypes = [_I64]
_lib.fp8blk_set_tensor_core_min_m.restype = _INT
_lib.fp8blk_set_tensor_core_min_m.argtypes = [_INT, _I64]
_lib.fp8blk_plan_query.restype = _INT
_lib.fp8blk_plan_query.argtypes = [_INT, _I64, _I64, _INT, _INT, _INT, _INT, _P]
_lib.fp8blk_device_status.restype = _INT
_lib.fp8blk_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), _INT]

# Return codes (include/fp8blk.h)
OK, EINVAL, EALIGN, ESCALE, EWS, ECUDA, ERANGE = 0, 1, 2, 3, 4, 5, 6
STATUS_WAIT_TIMEOUT = 1
STATUS_BAD_EXPERT = 2
STATUS_BAD_KV = 4
STATUS_KV_EXHAUSTED = 8
STATUS_BAD_TARGET = 16
MAX_M, MAX_HEAD_DIM, MAX_TOP, MAX_VOCAB = 8, 256, 32, 262144


class Fp8BlkError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {_lib.fp8blk_strerror(code).decode()} (code {code})")


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise Fp8BlkError(rc, where)


def _elsewhere(t: torch.Tensor, device: int, what: str = "a tensor") -> None:
    """Refuse a tensor that is not on the device (get_device() of the stream's tensor; the host is -1), unless it is pinned
    host memory, which kernels reach too: no pointer that a kernel could not follow is passed on."""
    if t.get_device() != device and not (t.device.type == "cpu" and t.is_pinned()):
        raise ValueError(f"{what} is on {t.device}, the call's other tensors are not")


def _ptr(t: torch.Tensor | None, device: int) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.get_device() != device:
        _elsewhere(t, device)
    return t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object around it


def _stream(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    return _raw_stream(t.get_device())


def abi_version() -> int:
    return _lib.fp8blk_abi_version()


# ---------------------------------------------------------------- host helper
def fp8blk_scales_from_e8m0(codes: np.ndarray | torch.Tensor) -> np.ndarray:
    """Decode an e8m0 scale grid on the host (same shape, float32)."""
    if isinstance(codes, torch.Tensor):
        codes = codes.cpu().numpy()
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    out = np.empty(codes.shape, dtype=np.float32)
    bad = ctypes.c_size_t(0)
    rc = _lib.fp8blk_scales_from_e8m0(codes.ctypes.data, codes.size, out.ctypes.data,
                                      ctypes.byref(bad))
    if rc == ESCALE:
        raise Fp8BlkError(rc, f"fp8blk_scales_from_e8m0 (flat index {bad.value})")
    _check(rc, "fp8blk_scales_from_e8m0")
    return out


# ---------------------------------------------------------------- GEMV
def fp8blk_gemv(w_codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                y: torch.Tensor | None = None) -> torch.Tensor:
    """y [m, rows] = decode(w_codes [rows, cols] e4m3 x scales [rows/128, cols/128]) @ x.T."""
    rows, cols = w_codes.shape
    x2 = x if x.dim() == 2 else x.view(1, -1)
    m = x2.shape[0]
    if y is None:
        y = torch.empty((m, rows), dtype=torch.float32, device=x.device)
    dev = x.get_device()
    _check(_lib.fp8blk_gemv(_ptr(w_codes, dev), _ptr(scales, dev), _ptr(x2, dev), _ptr(y, dev), m, rows, cols,
                            _stream(x)), "fp8blk_gemv")
    return y


def fp8blk_gemv_argmax_ws_bytes(m: int, rows: int, cols: int) -> int:
    return int(_lib.fp8blk_gemv_argmax_ws_bytes(m, rows, cols))


def argmax_workspace(m: int, rows: int, cols: int, device) -> torch.Tensor:
    """A zero-filled workspace of the size fp8blk_gemv_argmax needs."""
    n = fp8blk_gemv_argmax_ws_bytes(m, rows, cols)
    if n == 0:
        raise Fp8BlkError(EINVAL, "fp8blk_gemv_argmax_ws_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def fp8blk_gemv_argmax(w_codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                       ws: torch.Tensor, tokens: torch.Tensor | None = None,
                       logits: torch.Tensor | None = None) -> torch.Tensor:
    """Greedy tokens [m] (uint32 as int32 storage) of decode(W) @ x.T; logits optional."""
    rows, cols = w_codes.shape
    x2 = x if x.dim() == 2 else x.view(1, -1)
    m = x2.shape[0]
    if tokens is None:
        tokens = torch.empty(m, dtype=torch.int32, device=x.device)
    dev = x.get_device()
    _check(_lib.fp8blk_gemv_argmax(_ptr(w_codes, dev), _ptr(scales, dev), _ptr(x2, dev), _ptr(logits, dev),
                                   _ptr(tokens, dev), _ptr(ws, dev), ws.numel() * ws.element_size(), m,
                                   rows, cols, _stream(x)), "fp8blk_gemv_argmax")
    return tokens


def fp8blk_gemv_argmax_noalloc(w_codes: torch.Tensor, scales: torch.Tensor, x: torch.Tensor,
                               tokens: torch.Tensor | None = None,
                               logits: torch.Tensor | None = None) -> torch.Tensor:
    """fp8blk_gemv_argmax with the library's own fixed device scratch (no workspace).

    For callers that cannot allocate device memory; calls must not overlap on the GPU.
    """
    rows, cols = w_codes.shape
    x2 = x if x.dim() == 2 else x.view(1, -1)
    m = x2.shape[0]
    if tokens is None:
        tokens = torch.empty(m, dtype=torch.int32, device=x.device)
    dev = x.get_device()
    _check(_lib.fp8blk_gemv_argmax_noalloc(_ptr(w_codes, dev), _ptr(scales, dev), _ptr(x2, dev), _ptr(logits, dev),
                                           _ptr(tokens, dev), m, rows, cols, _stream(x)),
           "fp8blk_gemv_argmax_noalloc")
    return tokens


def fp8blk_bf16_gemv(w_bf16: torch.Tensor, x: torch.Tensor,
                     y: torch.Tensor | None = None) -> torch.Tensor:
    rows, cols = w_bf16.shape
    x2 = x if x.dim() == 2 else x.view(1, -1)
    m = x2.shape[0]
    if y is None:
        y = torch.empty((m, rows), dtype=torch.float32, device=x.device)
    dev = x.get_device()
    _check(_lib.fp8blk_bf16_gemv(_ptr(w_bf16, dev), _ptr(x2, dev), _ptr(y, dev), m, rows, cols, _stream(x)),
           "fp8blk_bf16_gemv")
    return y


# ---------------------------------------------------------------- NVFP4 experts
def _host_f32(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.cpu().numpy()
    return np.ascontiguousarray(a, dtype=np.float32)


def _host_i32(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.cpu().numpy()
    return np.ascontiguousarray(a, dtype=np.int32)


def nvfp4_expert_dequant(codes: torch.Tensor, scales: torch.Tensor, gscale, expert_id: int,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 bits (int16 storage) [rows, cols] of expert `expert_id`."""
    n_experts, rows, half = codes.shape
    cols = 2 * half
    g = _host_f32(gscale)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.int16, device=codes.device)
    dev = codes.get_device()
    _check(_lib.nvfp4_expert_dequant(_ptr(codes, dev), _ptr(scales, dev), g.ctypes.data, n_experts,
                                     int(expert_id), _ptr(out, dev), rows, cols, _stream(codes)),
           "nvfp4_expert_dequant")
    return out


def nvfp4_expert_dequant_gemv(codes: torch.Tensor, scales: torch.Tensor, gscale, ids,
                              x: torch.Tensor, scratch: torch.Tensor,
                              y: torch.Tensor | None = None) -> torch.Tensor:
    """y [n_active, rows]: each active expert dequantised into `scratch`, then GEMV'd."""
    n_experts, rows, half = codes.shape
    cols = 2 * half
    g = _host_f32(gscale)
    ids_h = _host_i32(ids)
    if y is None:
        y = torch.empty((ids_h.size, rows), dtype=torch.float32, device=x.device)
    dev = x.get_device()
    _check(_lib.nvfp4_expert_dequant_gemv(_ptr(codes, dev), _ptr(scales, dev), g.ctypes.data, n_experts,
                                          ids_h.ctypes.data, ids_h.size, _ptr(x, dev), _ptr(y, dev),
                                          _ptr(scratch, dev), rows, cols, _stream(x)),
           "nvfp4_expert_dequant_gemv")
    return y


def nvfp4_expert_gemv(codes: torch.Tensor, scales: torch.Tensor, gscale: torch.Tensor, ids: torch.Tensor,
                      x: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
    """y [n_active, rows] = W(ids[k]) x in one launch (CUDA cores or tensor
    cores, see set_fp4_kernel); `gscale` (f32 [n_experts]) and `ids` (int32
    [n_active]) stay on the device."""
    n_experts, rows, half = codes.shape
    cols = 2 * half
    if gscale.dtype != torch.float32 or ids.dtype != torch.int32:
        raise TypeError("gscale must be float32 and ids int32 device tensors")
    n_active = ids.numel()
    if y is None:
        y = torch.empty((n_active, rows), dtype=torch.float32, device=x.device)
    dev = x.get_device()
    _check(_lib.nvfp4_expert_gemv(_ptr(codes, dev), _ptr(scales, dev), _ptr(gscale, dev), n_experts, _ptr(ids, dev), n_active,
                                  _ptr(x, dev), _ptr(y, dev), rows, cols, _stream(x)), "nvfp4_expert_gemv")
    return y


def mxfp4_expert_gemv(codes: torch.Tensor, scales: torch.Tensor, ids: torch.Tensor, x: torch.Tensor,
                      y: torch.Tensor | None = None) -> torch.Tensor:
    """OCP MXFP4 experts: y [n_active, rows] = W(ids[k]) x in one launch
    (e8m0 scale per 32 columns; CUDA cores or tensor cores, see
    set_fp4_kernel; `ids` int32 on the device)."""
    n_experts, rows, half = codes.shape
    cols = 2 * half
    if ids.dtype != torch.int32:
        raise TypeError("ids must be an int32 device tensor")
    n_active = ids.numel()
    if y is None:
        y = torch.empty((n_active, rows), dtype=torch.float32, device=x.device)
    dev = x.get_device()
    _check(_lib.mxfp4_expert_gemv(_ptr(codes, dev), _ptr(scales, dev), n_experts, _ptr(ids, dev), n_active, _ptr(x, dev), _ptr(y, dev),
                                  rows, cols, _stream(x)), "mxfp4_expert_gemv")
    return y


# ---------------------------------------------------------------- paged cache
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    return code


def _typed(t: torch.Tensor, dtype: torch.dtype, what: str, device: int) -> int:
    """Data pointer of a contiguous tensor of exactly this type on this device (see _elsewhere)."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _refuse(t, dtype, what, device)
    return t.data_ptr()


def _refuse(t: torch.Tensor, dtype: torch.dtype, what: str, device: int) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    _elsewhere(t, device, what)
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _rows3(t: torch.Tensor, what: str, device: int) -> int:
    """Row stride of a [rows, heads, head_dim] tensor on this device whose rows are dense."""
    if t.get_device() != device:
        _elsewhere(t, device, what)
    if t.dim() != 3:
        raise ValueError(f"{what} must have 3 dimensions [rows, heads, head_dim]")
    rows, heads, dim = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise ValueError(f"{what}: heads and head_dim must be contiguous inside a row")
    return s0 if rows > 1 else heads * dim


_U8, _F32, _I32, _I64T = torch.uint8, torch.float32, torch.int32, torch.int64


def _cache(k_codes, k_scales, v_codes, v_scales, device):
    """Shape and data pointers of a cache: (n_blocks, kv_heads, block_tokens, head_dim), (k_codes, k_scales, ...)."""
    shape = k_codes.shape
    if len(shape) != 4 or v_codes.shape != shape:
        raise ValueError("k_codes and v_codes must both be [n_blocks, kv_heads, block_tokens, head_dim]")
    pairs = shape[:2]
    if k_scales.shape != pairs or v_scales.shape != pairs:
        raise ValueError("k_scales and v_scales must both be [n_blocks, kv_heads]")
    return shape, (_typed(k_codes, _U8, "k_codes", device), _typed(k_scales, _F32, "k_scales", device),
                   _typed(v_codes, _U8, "v_codes", device), _typed(v_scales, _F32, "v_scales", device))


class KvMap(NamedTuple):
    """What fp8blk_kv_map writes beside the block table."""
    seq_lens: torch.Tensor    # int32 [n]
    q_starts: torch.Tensor    # int32 [n + 1]
    slots: torch.Tensor       # int64 [max_tokens], -1 past the last new token
    positions: torch.Tensor   # int32 [max_tokens], -1 past the last new token
    free_head: torch.Tensor   # int32 [1], the next call's free_head


def kv_map_buffers(n: int, max_tokens: int, device) -> KvMap:
    """Output buffers of fp8blk_kv_map, for callers that keep them from step to step."""
    i32 = dict(dtype=torch.int32, device=device)
    return KvMap(torch.empty(n, **i32), torch.empty(n + 1, **i32),
                 torch.empty(max_tokens, dtype=torch.int64, device=device), torch.empty(max_tokens, **i32),
                 torch.empty(1, **i32))


def fp8blk_kv_map(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_blocks: torch.Tensor,
                  free_head: torch.Tensor, block_tokens: int, max_tokens: int, out: KvMap | None = None,
                  held: torch.Tensor | None = None, held_out: torch.Tensor | None = None) -> KvMap:
    """Block tables (updated in place), slots and positions of one step, from the requests' lengths on the device.

    Where tokens of earlier steps may have been rejected, `held` [n] counts the blocks that each request has (0 at first) and
    `held_out` [n], another tensor, receives the next step's counts, so that no block is taken twice."""
    n, width = block_table.shape
    if out is None:
        out = kv_map_buffers(n, max_tokens, block_table.device)
    if ctx_lens.numel() != n or new_lens.numel() != n or free_head.numel() != 1:
        raise ValueError("ctx_lens and new_lens must have one entry per row of block_table, free_head one")
    if (out.seq_lens.numel() != n or out.q_starts.numel() != n + 1 or out.slots.numel() != max_tokens
            or out.positions.numel() != max_tokens or out.free_head.numel() != 1):
        raise ValueError("out does not fit (see kv_map_buffers)")
    if (held is None) != (held_out is None) or (held is not None and (held.numel() != n or held_out.numel() != n)):
        raise ValueError("held and held_out go together, one entry each per row of block_table")
    i32, dev = torch.int32, block_table.get_device()
    rc = _lib.fp8blk_kv_map_held(_typed(ctx_lens, i32, "ctx_lens", dev), _typed(new_lens, i32, "new_lens", dev),
                                 None if held is None else _typed(held, i32, "held", dev),
                                 _typed(block_table, i32, "block_table", dev), _typed(free_blocks, i32, "free_blocks", dev),
                                 _typed(free_head, i32, "free_head", dev), _typed(out.seq_lens, i32, "out.seq_lens", dev),
                                 _typed(out.q_starts, i32, "out.q_starts", dev), _typed(out.slots, _I64T, "out.slots", dev),
                                 _typed(out.positions, i32, "out.positions", dev),
                                 _typed(out.free_head, i32, "out.free_head", dev),
                                 None if held_out is None else _typed(held_out, i32, "held_out", dev),
                                 n, width, free_blocks.numel(), block_tokens, max_tokens, _stream(block_table))
    if rc:
        _check(rc, "fp8blk_kv_map")
    return out


def fp8blk_kv_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor,
                     v_codes: torch.Tensor, v_scales: torch.Tensor) -> None:
    """Write keys and values [n, kv_heads, head_dim] (float32 or bfloat16; rows may be strided) into the cache at `slots`."""
    dev = k_codes.get_device()
    (blocks, heads, block, dim), cache = _cache(k_codes, k_scales, v_codes, v_scales, dev)
    n = slots.numel()
    if k.shape != (n, heads, dim) or v.shape != (n, heads, dim):
        raise ValueError("k and v must both be [len(slots), kv_heads, head_dim] of the cache")
    if v.dtype is not k.dtype:
        raise TypeError("k and v must have the same type")
    if n == 0:
        return
    rc = _lib.fp8blk_kv_append(k.data_ptr(), v.data_ptr(), _dtype(k, "k"), _typed(slots, _I64T, "slots", dev), *cache, n,
                               _rows3(k, "k", dev), _rows3(v, "v", dev), blocks, heads, block, dim, _stream(k_codes))
    if rc:
        _check(rc, "fp8blk_kv_append")


def fp8blk_kv_attn_ws_bytes(n_seqs: int, max_m: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_lib.fp8blk_kv_attn_ws_bytes(n_seqs, max_m, q_heads, kv_heads, head_dim))


def kv_attn_workspace(n_seqs: int, max_m: int, q_heads: int, kv_heads: int, head_dim: int, device) -> torch.Tensor:
    """A zero-filled workspace of the size fp8blk_kv_attn needs."""
    n = fp8blk_kv_attn_ws_bytes(n_seqs, max_m, q_heads, kv_heads, head_dim)
    if n == 0:
        raise Fp8BlkError(EINVAL, "fp8blk_kv_attn_ws_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def fp8blk_kv_attn(q: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                   v_scales: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor, q_starts: torch.Tensor,
                   max_m: int, sm_scale: float, ws: torch.Tensor, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of q [rows, q_heads, head_dim] (float32 or bfloat16; rows may be strided) over the paged cache; up to
    max_m rows per request.  `lse` (float32 [rows, q_heads]) is written when given."""
    dev = q.get_device()
    (blocks, kv_heads, block, dim), cache = _cache(k_codes, k_scales, v_codes, v_scales, dev)
    n, width = block_table.shape
    q_stride = _rows3(q, "q", dev)
    rows, q_heads, q_dim = q.shape
    if q_dim != dim:
        raise ValueError("q must be [rows, q_heads, head_dim] of the cache")
    if out is None:
        out = torch.empty((rows, q_heads, dim), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must have q's shape and type")
    if seq_lens.numel() != n or q_starts.numel() != n + 1:
        raise ValueError("seq_lens must have one entry per row of block_table, q_starts one more")
    if lse is not None and lse.shape != (rows, q_heads):
        raise ValueError("lse must be [rows, q_heads]")
    if rows == 0:
        return out
    rc = _lib.fp8blk_kv_attn(q.data_ptr(), _dtype(q, "q"), *cache, _typed(block_table, _I32, "block_table", dev),
                             _typed(seq_lens, _I32, "seq_lens", dev), _typed(q_starts, _I32, "q_starts", dev), out.data_ptr(),
                             None if lse is None else _typed(lse, _F32, "lse", dev), _typed(ws, ws.dtype, "ws", dev), ws.nbytes,
                             n, max_m, rows, q_heads, kv_heads, dim, block, blocks, width, q_stride, _rows3(out, "out", dev),
                             sm_scale, _stream(q))
    if rc:
        _check(rc, "fp8blk_kv_attn")
    return out


# ---------------------------------------------------------------- scoring
class TokenLogprobs(NamedTuple):
    """What fp8blk_token_logprobs writes."""
    logprob: torch.Tensor       # float32 [n]
    rank: torch.Tensor          # int32 [n]
    entropy: torch.Tensor       # float32 [n]
    top_ids: torch.Tensor       # int32 [n, top]
    top_logprobs: torch.Tensor  # float32 [n, top]


def token_logprobs_buffers(n: int, top: int, device) -> TokenLogprobs:
    """Output buffers of fp8blk_token_logprobs, for callers that keep them from step to step."""
    i32, f32 = dict(dtype=torch.int32, device=device), dict(dtype=torch.float32, device=device)
    return TokenLogprobs(torch.empty(n, **f32), torch.empty(n, **i32), torch.empty(n, **f32),
                         torch.empty((n, top), **i32), torch.empty((n, top), **f32))


def fp8blk_token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top: int = 0,
                          out: TokenLogprobs | None = None) -> TokenLogprobs:
    """Log probability, rank and entropy of `targets` [n] under logits [n, vocab] (float32 or bfloat16; rows may be
    strided), with the `top` most likely tokens."""
    if logits.dim() != 2 or targets.numel() != logits.shape[0]:
        raise ValueError("logits must be [n, vocab], targets [n]")
    n, vocab = logits.shape
    if logits.stride(1) != 1 and vocab > 1:
        raise ValueError("logits must be contiguous inside a row")
    if out is None:
        out = token_logprobs_buffers(n, top, logits.device)
    if out.logprob.numel() != n or out.rank.numel() != n or out.entropy.numel() != n or \
            out.top_ids.shape != (n, top) or out.top_logprobs.shape != (n, top):
        raise ValueError("out does not fit (see token_logprobs_buffers)")
    if n == 0:
        return out
    f32, i32, dev = torch.float32, torch.int32, logits.get_device()
    _check(_lib.fp8blk_token_logprobs(logits.data_ptr(), _dtype(logits, "logits"), _typed(targets, i32, "targets", dev),
                                      _typed(out.logprob, f32, "out.logprob", dev), _typed(out.rank, i32, "out.rank", dev),
                                      _typed(out.entropy, f32, "out.entropy", dev), _typed(out.top_ids, i32, "out.top_ids", dev),
                                      _typed(out.top_logprobs, f32, "out.top_logprobs", dev), n, vocab,
                                      logits.stride(0) if n > 1 else vocab, top, _stream(logits)),
           "fp8blk_token_logprobs")
    return out


# ---------------------------------------------------------------- control
def set_launch_tuning(target_stage_bytes: int = 0, ctas_per_sm: int = 0, use_pdl: int = 1,
                      l2_prefetch: int = 1, max_stages: int = 0) -> None:
    _check(_lib.fp8blk_set_launch_tuning(target_stage_bytes, ctas_per_sm, use_pdl, l2_prefetch,
                                         max_stages), "fp8blk_set_launch_tuning")


PLAN_FIELDS = ("panels", "panel_cols", "team_warps", "teams", "row_batches", "rows_per_batch",
               "stage_rows", "stage_bytes", "stages", "ctas_per_sm", "n_groups",
               "dynamic_smem_bytes", "kernel")


def plan_query(m: int, rows: int, cols: int, bytes_per_weight: int = 1, sms: int = 152,
               smem_per_sm: int = 233472, smem_per_block: int = 232448) -> dict:
    """Launch geometry for a shape on a device with the given facts (host only)."""
    out = np.zeros(13, dtype=np.int64)
    _check(_lib.fp8blk_plan_query(m, rows, cols, bytes_per_weight, sms, smem_per_sm,
                                  smem_per_block, out.ctypes.data), "fp8blk_plan_query")
    return dict(zip(PLAN_FIELDS, (int(v) for v in out)))


def set_m1_kernel(choice: int = 0, rowwarp_min_bytes: int = 0) -> None:
    """m = 1 kernel: 0 by size, 1 row-per-warp, 2 team (speed only)."""
    _check(_lib.fp8blk_set_m1_kernel(choice, rowwarp_min_bytes), "fp8blk_set_m1_kernel")


def set_fp4_kernel(choice: int = 0) -> None:
    """NVFP4 and MXFP4 expert GEMV kernel: 0 by shape (tensor cores from
    12288 active rows on), 1 CUDA cores, 2 tensor cores."""
    _check(_lib.fp8blk_set_fp4_kernel(choice), "fp8blk_set_fp4_kernel")


def set_tensor_core_min_m(min_m: int = 0, min_bytes: int = 0) -> None:
    """e4m3 GEMVs with m >= min_m (2..8; 9 = never) and at least min_bytes of
    weights (1 = any) run on the tensor cores; 0 restores a default."""
    _check(_lib.fp8blk_set_tensor_core_min_m(min_m, min_bytes), "fp8blk_set_tensor_core_min_m")


WAIT_LIMIT_DEFAULT_NS = 1_000_000_000


def set_wait_limit(limit_ns: int = WAIT_LIMIT_DEFAULT_NS) -> None:
    """How long a CUDA-core GEMV thread waits for a weight tile (or a role of fp8blk_kv_attn for its operands) before giving
    up (status FP8BLK_STATUS_WAIT_TIMEOUT); the default is about one second."""
    _check(_lib.fp8blk_set_wait_limit(int(limit_ns)), "fp8blk_set_wait_limit")


def fp8blk_device_status(clear: bool = False) -> int:
    """Device status word (0 = healthy).  Synchronizes the current device."""
    v = ctypes.c_uint32(0)
    _check(_lib.fp8blk_device_status(ctypes.byref(v), int(clear)), "fp8blk_device_status")
    return int(v.value)


def raw_library() -> ctypes.CDLL:
    """The loaded ctypes library, for callers that pass raw pointers."""
    return _lib
