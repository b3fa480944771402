"""int4 KV-cache quantize-on-store and fused decode attention for GB300.

Thin Python binding over the C-ABI library ``libtq.so`` (see include/tq.h):
argument marshalling only.  Every step of the path runs in the library's CUDA
kernels; PyTorch supplies device memory and the current stream.  There is no
fallback: if the compiled library is missing, every entry point raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

__all__ = [
    "TQ_OK", "TQ_IMPL_AUTO", "TQ_IMPL_MMA", "TQ_IMPL_SIMT", "TQ_DEV_WRITE_POS", "TQ_DEV_SEQ_LEN",
    "TQ_DEV_TIMEOUT", "TQError", "lib", "lib_path", "tq_kv_cache", "KVCache",
    "tq_abi_version", "tq_status_string", "tq_kv_cache_bytes", "tq_sdpa_workspace_bytes", "workspace",
    "tq_quantize_kv_append", "tq_sdpa_int4_decode", "tq_sdpa_int4_partial", "tq_sdpa_int4_reduce",
    "tq_sdpa_plan", "tq_split_plan", "tq_sdpa_int4_decode_noalloc", "NOALLOC_SCRATCH_BYTES", "tq_decode_step",
    "tq_dequantize_kv", "tq_hadamard_rotate", "TQ_ROTATE_K", "TQ_ROTATE_V", "TQ_STEP_ADVANCE", "TQ_DEV_PAGE",
    "tq_paged_kv_cache", "PagedKVCache", "tq_decode_step_host", "tq_host_staging_bytes",
    "TQ_DEV_BLOCK", "TQ_ROPE_PAIRS", "TQ_ROPE_INVERSE", "tq_rope_axes", "block_bounds", "tq_kv_block_bounds",
    "sparse_workspace", "tq_select_blocks", "tq_sdpa_blocks_decode", "tq_sparse_decode", "weights_workspace",
    "tq_sdpa_decode_weights", "tq_kv_evict",
]

TQ_OK = 0
TQ_IMPL_AUTO, TQ_IMPL_MMA, TQ_IMPL_SIMT = 0, 1, 2
TQ_DEV_WRITE_POS, TQ_DEV_SEQ_LEN, TQ_DEV_TIMEOUT = 0x1, 0x2, 0x4
TQ_ROTATE_K, TQ_ROTATE_V = 0x1, 0x2
TQ_STEP_ADVANCE = 0x100
TQ_DEV_PAGE = 0x8
TQ_DEV_BLOCK = 0x10
TQ_ROPE_PAIRS, TQ_ROPE_INVERSE = 0x1, 0x2
GROUP_SIZE = 64
DEFAULT_CHUNK = 512
NOALLOC_SCRATCH_BYTES = 4 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "_build", "libtq.so")


class TQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().tq_status_string(status).decode()
        if status == 5:
            msg += f" (cudaError {lib().tq_last_cuda_error()})"
        super().__init__(f"{fn}: {msg} [status {status}]")
        self.status = status


class tq_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("k_bias", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("v_bias", ctypes.c_void_p),
        ("batch", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32),
        ("capacity", ctypes.c_int32), ("bits", ctypes.c_int32),
    ]


class tq_paged_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("k_bias", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("v_bias", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("batch", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32), ("bits", ctypes.c_int32),
    ]


class tq_rope_rows(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("stride_b", ctypes.c_int64), ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64),
        ("num_heads", ctypes.c_int32),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libtq.so (built by ``build.build()``); raises if it is not there."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError(f"libtq.so not built ({path}); run int4_kv_cache_gb300.build.build()")
        L = ctypes.CDLL(path)
        P, i32, sz, f32, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float, ctypes.c_uint32
        C = ctypes.POINTER(tq_kv_cache)
        PC = ctypes.POINTER(tq_paged_kv_cache)
        sig = {
            "tq_abi_version": ([], i32),
            "tq_status_string": ([i32], ctypes.c_char_p),
            "tq_last_cuda_error": ([], i32),
            "tq_wait_timeout_selftest": ([P, P, u32, P, P], i32),
            "tq_kv_cache_bytes": ([i32] * 5, sz),
            "tq_kv_cache_carve": ([C, P, i32, i32, i32, i32, i32], i32),
            "tq_quantize_kv_append": ([C, P, P, i32, P, P, P], i32),
            "tq_sdpa_workspace_bytes": ([i32] * 6, sz),
            "tq_sdpa_int4_decode": ([C, P, i32, P, i32, f32, i32, P, sz, P, P, P], i32),
            "tq_sdpa_int4_decode_impl": ([C, P, i32, P, i32, f32, i32, P, sz, P, P, i32, P], i32),
            "tq_sdpa_plan": ([C, i32, i32, i32, i32, P, P], i32),
            "tq_split_plan": ([i32, i32, i32, i32, i32, i32, i32, P, P], i32),
            "tq_sdpa_int4_partial": ([C, P, i32, P, i32, f32, i32, i32, P, P, P, P, i32, P], i32),
            "tq_sdpa_int4_reduce": ([P, P, P, i32, i32, i32, i32, P, P], i32),
            "tq_sdpa_int4_decode_noalloc": ([C, P, i32, P, i32, f32, i32, P, P, P], i32),
            "tq_decode_step": ([C, P, P, i32, P, P, i32, P, i32, f32, i32, P, sz, P, P, P], i32),
            "tq_dequantize_kv": ([C, i32, P, P, P], i32),
            "tq_quantize_kv_append_ex": ([C, P, P, i32, P, u32, P, P], i32),
            "tq_hadamard_rotate": ([P, ctypes.c_int64, i32, P, P], i32),
            "tq_sdpa_int4_decode_ex": ([C, P, i32, P, i32, f32, i32, u32, P, sz, P, P, P], i32),
            "tq_decode_step_ex": ([C, P, P, i32, P, P, i32, P, i32, f32, i32, u32, P, sz, P, P, P], i32),
            "tq_paged_kv_cache_bytes": ([i32] * 6, sz),
            "tq_paged_kv_cache_carve": ([PC, P, P] + [i32] * 8, i32),
            "tq_kv_cache_bytes_ex": ([i32] * 6, sz),
            "tq_host_staging_bytes": ([i32] * 5, sz),
            "tq_decode_step_host": ([C, P, P, i32, P, P, i32, P, i32, f32, i32, u32, P, sz, P, sz, P, P, P], i32),
            "tq_kv_cache_carve_ex": ([C, P] + [i32] * 6, i32),
            "tq_paged_quantize_kv_append": ([PC, P, P, i32, P, u32, P, P], i32),
            "tq_paged_sdpa_int4_decode": ([PC, P, i32, P, i32, f32, i32, u32, P, sz, P, P, P], i32),
            "tq_paged_decode_step": ([PC, P, P, i32, P, P, i32, P, i32, f32, i32, u32, P, sz, P, P, P], i32),
        }
        R = ctypes.POINTER(tq_rope_rows)
        for pre, cache in (("tq_", C), ("tq_paged_", PC)):
            sig[pre + "kv_block_bounds"] = ([cache, i32, P, i32, P, P, P], i32)
            sig[pre + "sdpa_blocks_decode"] = ([cache, P, i32, P, i32, f32, P, i32, i32, u32, P, sz, P, P, P], i32)
            sig[pre + "sparse_decode"] = ([cache, P, P, i32, P, i32, f32, i32, i32, i32, i32, u32, P, sz, P, P, P, P], i32)
            sig[pre + "sdpa_decode_weights"] = ([cache, P, i32, P, i32, f32, f32, P, u32, P, sz, P, P, P], i32)
            sig[pre + "kv_evict"] = ([cache, cache, P, P, i32, i32, i32, P, P, P, P, P], i32)
        sig["tq_rope_axes"] = ([R, R, P, P, i32, P, i32, i32, i32, i32, u32, P], i32)
        sig["tq_block_bounds_bytes"] = ([i32] * 5, sz)
        sig["tq_sparse_workspace_bytes"] = ([i32] * 7, sz)
        sig["tq_select_blocks"] = ([P, P] + [i32] * 5 + [P] + [i32] * 5 + [u32, P, sz, P, P, P], i32)
        sig["tq_weights_workspace_bytes"] = ([i32] * 5, sz)
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        if L.tq_abi_version() != 2:
            raise ImportError("libtq.so ABI version mismatch")
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != TQ_OK:
        raise TQError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: Optional[torch.cuda.Stream]):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is not None:  # the current stream's handle without building a Stream object
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """An output that a call on ``stream`` makes.  On another stream than the current one it is that stream's memory (memory of
    the current one may still be in use there by what its last owner queued), kept until the current stream, where the caller
    goes on with it, is past its use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(out.device))
    return out


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")


# ------------------------------------------------------------------ host-only
def tq_abi_version() -> int:
    return int(lib().tq_abi_version())


def tq_wait_timeout_selftest(src: torch.Tensor, status: torch.Tensor, limit_us: int, copied: torch.Tensor,
                             stream=None) -> None:
    """The bounded-wait diagnostic: a 1 KB copy from ``src`` (uint8, >= 1024
    bytes), then a wait nothing ends, given up after ``limit_us``."""
    _need(src, torch.uint8, "src")
    _need(status, torch.int32, "status")
    _need(copied, torch.int32, "copied")
    if src.numel() < 1024:
        raise ValueError("src must hold at least 1024 bytes")
    _check("tq_wait_timeout_selftest", lib().tq_wait_timeout_selftest(_ptr(src), _ptr(status), int(limit_us),
                                                                      _ptr(copied), _stream(stream)))


def tq_status_string(status: int) -> str:
    return lib().tq_status_string(status).decode()


def tq_kv_cache_bytes(batch: int, num_kv_heads: int, head_dim: int, group_size: int, capacity: int) -> int:
    return int(lib().tq_kv_cache_bytes(batch, num_kv_heads, head_dim, group_size, capacity))


def tq_sdpa_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
                            chunk: int = DEFAULT_CHUNK) -> int:
    return int(lib().tq_sdpa_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, chunk))


def workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
              chunk: int = DEFAULT_CHUNK, device="cuda") -> torch.Tensor:
    """A decode workspace of tq_sdpa_workspace_bytes bytes (zero-filled)."""
    return torch.zeros(tq_sdpa_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, chunk),
                       dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ the cache
class KVCache:
    """One layer's int4 cache in a single device allocation (torch uint8).

    Views: k_codes/v_codes uint8 [B, Hkv, cap, D/2]; k_scale/k_bias/v_scale/v_bias
    fp16 [B, Hkv, cap, D/64].  ``struct`` is the tq_kv_cache handed to the ABI.
    """

    paged = False

    def __init__(self, batch: int, num_kv_heads: int, head_dim: int, capacity: int,
                 device=None, group_size: int = GROUP_SIZE, bits: int = 4):
        nbytes = int(lib().tq_kv_cache_bytes_ex(batch, num_kv_heads, head_dim, group_size, bits, capacity))
        if nbytes == 0:
            raise ValueError("invalid cache sizes")
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
        self.struct = tq_kv_cache()
        _check("tq_kv_cache_carve_ex", lib().tq_kv_cache_carve_ex(ctypes.byref(self.struct), _ptr(self.buffer),
                                                                   batch, num_kv_heads, head_dim, group_size, bits,
                                                                   capacity))
        self.batch, self.num_kv_heads, self.head_dim, self.capacity = batch, num_kv_heads, head_dim, capacity
        self.group_size, self.bits = group_size, bits
        base = self.buffer.data_ptr()
        rows = batch * num_kv_heads * capacity
        ng = head_dim // group_size

        def view(addr, n, dtype, shape):
            off = addr - base
            nb = n * torch.empty((), dtype=dtype).element_size()
            return self.buffer[off: off + nb].view(dtype).view(shape)

        cw = head_dim * bits // 8
        cs = (batch, num_kv_heads, capacity, cw)
        ss = (batch, num_kv_heads, capacity, ng)
        s = self.struct
        self.k_codes = view(s.k_codes, rows * cw, torch.uint8, cs)
        self.v_codes = view(s.v_codes, rows * cw, torch.uint8, cs)
        self.k_scale = view(s.k_scale, rows * ng, torch.float16, ss)
        self.k_bias = view(s.k_bias, rows * ng, torch.float16, ss)
        self.v_scale = view(s.v_scale, rows * ng, torch.float16, ss)
        self.v_bias = view(s.v_bias, rows * ng, torch.float16, ss)

    @property
    def nbytes(self) -> int:
        return self.buffer.numel()

    def ref(self):
        return ctypes.byref(self.struct)


class PagedKVCache:
    """A page pool (one device allocation) plus a device block table.

    Views: k_codes/v_codes uint8 [num_pages, Hkv, page_tokens, D/2];
    k_scale/k_bias/v_scale/v_bias fp16 [num_pages, Hkv, page_tokens, D/64];
    block_table int32 [B, max_pages_per_seq] (the caller fills it: page of
    logical page j of sequence b).  Every call of this binding that takes a
    ``KVCache`` takes a ``PagedKVCache`` as well.
    """

    paged = True

    def __init__(self, batch: int, num_kv_heads: int, head_dim: int, page_tokens: int, num_pages: int,
                 max_pages_per_seq: int, device=None, group_size: int = GROUP_SIZE, bits: int = 4):
        nbytes = int(lib().tq_paged_kv_cache_bytes(num_pages, num_kv_heads, head_dim, group_size, bits, page_tokens))
        if nbytes == 0:
            raise ValueError("invalid page pool sizes")
        dev = device or "cuda"
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.block_table = torch.zeros((batch, max_pages_per_seq), dtype=torch.int32, device=dev)
        self.struct = tq_paged_kv_cache()
        _check("tq_paged_kv_cache_carve", lib().tq_paged_kv_cache_carve(
            ctypes.byref(self.struct), _ptr(self.buffer), _ptr(self.block_table), batch, num_kv_heads, head_dim,
            group_size, bits, page_tokens, num_pages, max_pages_per_seq))
        self.batch, self.num_kv_heads, self.head_dim = batch, num_kv_heads, head_dim
        self.page_tokens, self.num_pages, self.max_pages_per_seq = page_tokens, num_pages, max_pages_per_seq
        self.capacity = page_tokens * max_pages_per_seq
        self.group_size, self.bits = group_size, bits
        base = self.buffer.data_ptr()
        rows = num_pages * num_kv_heads * page_tokens
        ng = head_dim // group_size

        def view(addr, n, dtype, shape):
            off = addr - base
            nb = n * torch.empty((), dtype=dtype).element_size()
            return self.buffer[off: off + nb].view(dtype).view(shape)

        cw = head_dim * bits // 8
        cs = (num_pages, num_kv_heads, page_tokens, cw)
        ss = (num_pages, num_kv_heads, page_tokens, ng)
        st = self.struct
        self.k_codes = view(st.k_codes, rows * cw, torch.uint8, cs)
        self.v_codes = view(st.v_codes, rows * cw, torch.uint8, cs)
        self.k_scale = view(st.k_scale, rows * ng, torch.float16, ss)
        self.k_bias = view(st.k_bias, rows * ng, torch.float16, ss)
        self.v_scale = view(st.v_scale, rows * ng, torch.float16, ss)
        self.v_bias = view(st.v_bias, rows * ng, torch.float16, ss)

    def ref(self):
        return ctypes.byref(self.struct)


# ------------------------------------------------------------------ device ops
def tq_quantize_kv_append(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, write_pos: torch.Tensor,
                          status: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> None:
    """Quantize k_new/v_new [B, Hkv, n_new, D] fp16 into cache rows write_pos[b] + i
    (flags TQ_ROTATE_K / TQ_ROTATE_V: Hadamard-rotate the rows first)."""
    _need(k_new, torch.float16, "k_new")
    _need(v_new, torch.float16, "v_new")
    _need(write_pos, torch.int32, "write_pos")
    if status is not None:
        _need(status, torch.int32, "status")
    n_new = k_new.shape[2] if k_new.dim() == 4 else 0
    if tuple(k_new.shape) != (cache.batch, cache.num_kv_heads, n_new, cache.head_dim) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new/v_new must be [B, Hkv, n_new, D]; got {tuple(k_new.shape)}")
    if getattr(cache, "paged", False):
        _check("tq_paged_quantize_kv_append", lib().tq_paged_quantize_kv_append(
            cache.ref(), _ptr(k_new), _ptr(v_new), n_new, _ptr(write_pos), int(flags), _ptr(status), _stream(stream)))
        return
    if flags:
        _check("tq_quantize_kv_append_ex", lib().tq_quantize_kv_append_ex(
            cache.ref(), _ptr(k_new), _ptr(v_new), n_new, _ptr(write_pos), int(flags), _ptr(status), _stream(stream)))
        return
    _check("tq_quantize_kv_append", lib().tq_quantize_kv_append(cache.ref(), _ptr(k_new), _ptr(v_new), n_new,
                                                                _ptr(write_pos), _ptr(status), _stream(stream)))


def tq_sdpa_int4_decode(cache: KVCache, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                        attn_scale: float, workspace: torch.Tensor, out: Optional[torch.Tensor] = None,
                        chunk: int = DEFAULT_CHUNK, status: Optional[torch.Tensor] = None,
                        impl: int = TQ_IMPL_AUTO, stream=None, flags: int = 0) -> torch.Tensor:
    """Fused int4 decode attention; q [B, Hq, D] fp16 -> out [B, Hq, D] fp16
    (flags: the rotation flags the cache was written with)."""
    _need(q, torch.float16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(workspace, torch.uint8, "workspace")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q.dtype, q.device, stream)
    _need(out, torch.float16, "out")
    if status is not None:
        _need(status, torch.int32, "status")
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cache.head_dim or out.shape != q.shape:
        raise ValueError(f"q must be [B, Hq, D]; got {tuple(q.shape)}")
    if getattr(cache, "paged", False):
        if impl == TQ_IMPL_SIMT:
            raise ValueError("a paged cache takes the tensor-core implementation")
        _check("tq_paged_sdpa_int4_decode", lib().tq_paged_sdpa_int4_decode(
            cache.ref(), _ptr(q), q.shape[1], _ptr(seq_lens), int(max_seq_len), float(attn_scale), int(chunk),
            int(flags), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(status), _stream(stream)))
        return out
    if flags:
        if impl != TQ_IMPL_AUTO:
            raise ValueError("rotation flags take the default implementation")
        _check("tq_sdpa_int4_decode_ex", lib().tq_sdpa_int4_decode_ex(
            cache.ref(), _ptr(q), q.shape[1], _ptr(seq_lens), int(max_seq_len), float(attn_scale), int(chunk),
            int(flags), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(status), _stream(stream)))
        return out
    _check("tq_sdpa_int4_decode", lib().tq_sdpa_int4_decode_impl(
        cache.ref(), _ptr(q), q.shape[1], _ptr(seq_lens), int(max_seq_len), float(attn_scale), int(chunk),
        _ptr(workspace), workspace.numel(), _ptr(out), _ptr(status), int(impl), _stream(stream)))
    return out


def tq_decode_step(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, write_pos: torch.Tensor,
                   q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, attn_scale: float,
                   workspace: torch.Tensor, out: Optional[torch.Tensor] = None, chunk: int = DEFAULT_CHUNK,
                   status: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> torch.Tensor:
    """Append k_new/v_new [B, Hkv, n_new, D] at write_pos, then decode q [B, Hq, D]
    over seq_lens (which must already count the new tokens); flags: rotation."""
    for t, n, dt in ((k_new, "k_new", torch.float16), (v_new, "v_new", torch.float16), (q, "q", torch.float16),
                     (write_pos, "write_pos", torch.int32), (seq_lens, "seq_lens", torch.int32),
                     (workspace, "workspace", torch.uint8)):
        _need(t, dt, n)
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q.dtype, q.device, stream)
    _need(out, torch.float16, "out")
    if status is not None:
        _need(status, torch.int32, "status")
    n_new = k_new.shape[2] if k_new.dim() == 4 else 0
    if tuple(k_new.shape) != (cache.batch, cache.num_kv_heads, n_new, cache.head_dim) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new/v_new must be [B, Hkv, n_new, D]; got {tuple(k_new.shape)}")
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cache.head_dim or out.shape != q.shape:
        raise ValueError(f"q must be [B, Hq, D]; got {tuple(q.shape)}")
    if getattr(cache, "paged", False):
        _check("tq_paged_decode_step", lib().tq_paged_decode_step(
            cache.ref(), _ptr(k_new), _ptr(v_new), n_new, _ptr(write_pos), _ptr(q), q.shape[1], _ptr(seq_lens),
            int(max_seq_len), float(attn_scale), int(chunk), int(flags), _ptr(workspace), workspace.numel(),
            _ptr(out), _ptr(status), _stream(stream)))
        return out
    if flags:
        _check("tq_decode_step_ex", lib().tq_decode_step_ex(
            cache.ref(), _ptr(k_new), _ptr(v_new), n_new, _ptr(write_pos), _ptr(q), q.shape[1], _ptr(seq_lens),
            int(max_seq_len), float(attn_scale), int(chunk), int(flags), _ptr(workspace), workspace.numel(),
            _ptr(out), _ptr(status), _stream(stream)))
        return out
    _check("tq_decode_step", lib().tq_decode_step(
        cache.ref(), _ptr(k_new), _ptr(v_new), n_new, _ptr(write_pos), _ptr(q), q.shape[1], _ptr(seq_lens),
        int(max_seq_len), float(attn_scale), int(chunk), _ptr(workspace), workspace.numel(), _ptr(out),
        _ptr(status), _stream(stream)))
    return out


def tq_sdpa_plan(cache: KVCache, num_q_heads: int, max_seq_len: int, chunk: int = DEFAULT_CHUNK,
                 impl: int = TQ_IMPL_AUTO):
    """(n_splits, max_run_tokens) of the runs tq_sdpa_int4_decode uses on this device."""
    ns, run = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("tq_sdpa_plan", lib().tq_sdpa_plan(cache.ref(), num_q_heads, int(max_seq_len), int(chunk), int(impl),
                                              ctypes.byref(ns), ctypes.byref(run)))
    return ns.value, run.value


def tq_split_plan(batch: int, num_kv_heads: int, max_seq_len: int, chunk: int, tile_tokens: int,
                  resident_ctas: int, merge: bool = True):
    """(n_splits, max_run_tokens) of the split rule for a device holding
    ``resident_ctas`` phase-1 CTAs at once (host arithmetic, no device);
    ``merge``: the decode may merge its runs itself (no reduce)."""
    ns, run = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("tq_split_plan", lib().tq_split_plan(int(batch), int(num_kv_heads), int(max_seq_len), int(chunk),
                                                int(tile_tokens), int(resident_ctas), int(bool(merge)),
                                                ctypes.byref(ns), ctypes.byref(run)))
    return ns.value, run.value


def tq_sdpa_int4_partial(cache: KVCache, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                         attn_scale: float, chunk: int = DEFAULT_CHUNK, chunks_per_split: int = 1,
                         status: Optional[torch.Tensor] = None, impl: int = TQ_IMPL_AUTO, stream=None,
                         out=None):
    """Phase 1 alone: (m, l, acc) fp32 per part of ``chunks_per_split`` chunks
    (1 = per chunk; 0 = the runs tq_sdpa_int4_decode uses), m in natural-log units."""
    _need(q, torch.float16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    B, Hq, D = q.shape
    nc = max(1, math.ceil(max_seq_len / chunk))
    if chunks_per_split > 0:
        n_parts = math.ceil(nc / chunks_per_split)
    else:
        n_parts = tq_sdpa_plan(cache, Hq, max_seq_len, chunk, impl)[0]
    if out is None:
        m, l = (_new((B, Hq, n_parts), torch.float32, q.device, stream) for _ in range(2))
        acc = _new((B, Hq, n_parts, D), torch.float32, q.device, stream)
    else:
        m, l, acc = out
        if m.numel() < B * Hq * n_parts or acc.numel() < B * Hq * n_parts * D:
            raise ValueError("partial output buffers too small")
    _check("tq_sdpa_int4_partial", lib().tq_sdpa_int4_partial(
        cache.ref(), _ptr(q), Hq, _ptr(seq_lens), int(max_seq_len), float(attn_scale), int(chunk),
        int(chunks_per_split),
        _ptr(m), _ptr(l), _ptr(acc), _ptr(status), int(impl), _stream(stream)))
    return m, l, acc


def tq_sdpa_int4_reduce(m: torch.Tensor, l: torch.Tensor, acc: torch.Tensor, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Phase 2 alone: LSE merge of [B, Hq, n] partials -> fp16 [B, Hq, D]."""
    for t, n in ((m, "m"), (l, "l"), (acc, "acc")):
        _need(t, torch.float32, n)
    B, Hq, n, D = acc.shape
    if out is None:
        out = _new((B, Hq, D), torch.float16, acc.device, stream)
    _need(out, torch.float16, "out")
    _check("tq_sdpa_int4_reduce", lib().tq_sdpa_int4_reduce(_ptr(m), _ptr(l), _ptr(acc), B, Hq, D, n, _ptr(out),
                                                            _stream(stream)))
    return out


def tq_sdpa_int4_decode_noalloc(cache: KVCache, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                                attn_scale: float, out: Optional[torch.Tensor] = None, chunk: int = DEFAULT_CHUNK,
                                status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tq_sdpa_int4_decode without a workspace: the partial states live in a
    fixed 4 MiB device array owned by the library (for callers that cannot
    allocate).  Calls that overlap on the GPU share that array and race."""
    _need(q, torch.float16, "q")
    _need(seq_lens, torch.int32, "seq_lens")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q.dtype, q.device, stream)
    _need(out, torch.float16, "out")
    if status is not None:
        _need(status, torch.int32, "status")
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cache.head_dim or out.shape != q.shape:
        raise ValueError(f"q must be [B, Hq, D]; got {tuple(q.shape)}")
    _check("tq_sdpa_int4_decode_noalloc", lib().tq_sdpa_int4_decode_noalloc(
        cache.ref(), _ptr(q), q.shape[1], _ptr(seq_lens), int(max_seq_len), float(attn_scale), int(chunk),
        _ptr(out), _ptr(status), _stream(stream)))
    return out


def tq_dequantize_kv(cache: KVCache, n_rows: int, out=None, stream=None):
    """fp16 K and V [B, Hkv, n_rows, D] of rows [0, n_rows) of the cache:
    fp16_rne(fp32(scale * code + bias)).  The float cache of the
    dequantize-then-attend comparison path; the fused decode never uses it."""
    shape = (cache.batch, cache.num_kv_heads, int(n_rows), cache.head_dim)
    if out is None:
        dev = cache.buffer.device
        out = (_new(shape, torch.float16, dev, stream), _new(shape, torch.float16, dev, stream))
    k, v = out
    for t, n in ((k, "k_out"), (v, "v_out")):
        _need(t, torch.float16, n)
        if tuple(t.shape) != shape:
            raise ValueError(f"{n} must be {shape}; got {tuple(t.shape)}")
    _check("tq_dequantize_kv", lib().tq_dequantize_kv(cache.ref(), int(n_rows), _ptr(k), _ptr(v), _stream(stream)))
    return k, v


def tq_hadamard_rotate(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp16 rows [..., D] (D = 64, 128, 256) -> fp16_rne(H x) per row, H the
    normalised Sylvester Hadamard matrix (out may be x)."""
    _need(x, torch.float16, "x")
    if out is None:
        out = torch.empty_like(x) if stream is None else _new(x.shape, x.dtype, x.device, stream)
    _need(out, torch.float16, "out")
    if out.shape != x.shape:
        raise ValueError("out must have the shape of x")
    dim = x.shape[-1]
    _check("tq_hadamard_rotate", lib().tq_hadamard_rotate(_ptr(x), x.numel() // dim, dim, _ptr(out),
                                                          _stream(stream)))
    return out


def tq_host_staging_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, n_new: int) -> int:
    return int(lib().tq_host_staging_bytes(batch, num_q_heads, num_kv_heads, head_dim, n_new))


def _need_host(t: torch.Tensor, name: str) -> None:
    if t.is_cuda or t.dtype != torch.float16 or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous host float16 tensor (pinned for asynchronous copies)")


def tq_decode_step_host(cache: KVCache, h_k_new: torch.Tensor, h_v_new: torch.Tensor, write_pos: torch.Tensor,
                        h_q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, attn_scale: float,
                        workspace: torch.Tensor, staging: torch.Tensor, h_out: torch.Tensor,
                        chunk: int = DEFAULT_CHUNK, flags: int = 0, status: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """tq_decode_step with q / k_new / v_new / out in host memory: the copies and
    the step are queued by one library call; h_out is valid once the stream
    has reached it."""
    for t, n in ((h_k_new, "h_k_new"), (h_v_new, "h_v_new"), (h_q, "h_q"), (h_out, "h_out")):
        _need_host(t, n)
    for t, n, dt in ((write_pos, "write_pos", torch.int32), (seq_lens, "seq_lens", torch.int32),
                     (workspace, "workspace", torch.uint8), (staging, "staging", torch.uint8)):
        _need(t, dt, n)
    n_new = h_k_new.shape[2] if h_k_new.dim() == 4 else 0
    _check("tq_decode_step_host", lib().tq_decode_step_host(
        cache.ref(), _ptr(h_k_new), _ptr(h_v_new), n_new, _ptr(write_pos), _ptr(h_q), h_q.shape[1], _ptr(seq_lens),
        int(max_seq_len), float(attn_scale), int(chunk), int(flags), _ptr(workspace), workspace.numel(),
        _ptr(staging), staging.numel(), _ptr(h_out), _ptr(status), _stream(stream)))
    return h_out


# ------------------------------------------------- rotary positions, sparse decode, eviction
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(stream, *tensors):
    """The handle of the stream to use (None: the current one); all tensors on one device, the current one (the kernels
    run there)."""
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"a tensor on {t.device}, but the current device is cuda:{dev}")
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _rope_rows(x: torch.Tensor, out: Optional[torch.Tensor], b: int, n: int, d: int, stream, name: str):
    """(the rows as the library takes them, their output [B, heads, n, D])."""
    if not x.is_cuda or x.dtype != torch.float16 or x.stride(3) != 1:
        raise ValueError(f"{name}: expected a CUDA float16 tensor [B, n, heads, D] with a contiguous last dimension")
    h = x.shape[2]
    if out is None:
        shape = (b, h, n, d)
        out = torch.empty(shape, dtype=torch.float16, device=x.device) if stream is None else _new(shape, torch.float16, x.device, stream)
    else:
        _need(out, torch.float16, name + "_out")
        if out.shape != (b, h, n, d):
            raise ValueError(f"{name}_out must be [B, heads, n, D] = {(b, h, n, d)}; got {tuple(out.shape)}")
    sb, st, sh, _ = x.stride()
    # a dimension of one is never stepped along, whatever its stride says
    return tq_rope_rows(x.data_ptr(), out.data_ptr(), sb if b > 1 else 0, st if n > 1 else 0, sh if h > 1 else 0, h), out


def tq_rope_axes(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor, sections,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, flags: int = 0, stream=None):
    """Rotary positions with several axes: q [B, n, Hq, D] and k [B, n, Hkv, D]
    (or None) fp16, any strides of whole 8-element steps, -> [B, Hq, n, D] and
    [B, Hkv, n, D].  positions int32 [axes, B, n]; inv_freq fp32
    [rotary_dim / 2]; sections: how many of the pairs follow each axis.  flags:
    TQ_ROPE_PAIRS (neighbouring elements form a pair), TQ_ROPE_INVERSE (turn back;
    the gradient of the rows)."""
    _need(positions, torch.int32, "positions")
    _need(inv_freq, torch.float32, "inv_freq")
    if q.dim() != 4:
        raise ValueError(f"q must be [B, n, Hq, D]; got {tuple(q.shape)}")
    b, n, _, d = q.shape
    if k is not None and (k.dim() != 4 or k.shape != (b, n, k.shape[2], d)):
        raise ValueError(f"k must be [B, n, Hkv, D] with q's B, n and D; got {tuple(k.shape)}")
    if positions.shape != (len(sections), b, n):
        raise ValueError(f"positions must be [axes, B, n] = {(len(sections), b, n)}; got {tuple(positions.shape)}")
    rq, q_out = _rope_rows(q, q_out, b, n, d, stream, "q")
    rk = None
    if k is not None:
        rk, k_out = _rope_rows(k, k_out, b, n, d, stream, "k")
    on = _on(stream, q, k, positions, inv_freq, q_out, k_out)
    if n > 0:
        _check("tq_rope_axes", lib().tq_rope_axes(rq, rk, positions.data_ptr(), inv_freq.data_ptr(), len(sections),
                                                  (ctypes.c_int32 * len(sections))(*sections), b, n, d, 2 * inv_freq.numel(),
                                                  int(flags), on))
    return (q_out, k_out) if k is not None else q_out


_layout_fns = {}


def _fn(cache, name: str):
    """The entry point of the cache's layout."""
    fns = _layout_fns.get(name)
    if fns is None:
        fns = _layout_fns[name] = (getattr(lib(), "tq_" + name), getattr(lib(), "tq_paged_" + name))
    return fns[cache.paged]


def _block_count(capacity: int, block_tokens: int) -> int:
    if block_tokens not in (32, 64, 128):
        raise ValueError(f"block_tokens must be 32, 64 or 128; got {block_tokens}")
    return -(-int(capacity) // block_tokens)


def block_bounds(cache, block_tokens: int = 64) -> torch.Tensor:
    """The bounds of every block of a cache, fp16 [B, Hkv, ceil(capacity / block_tokens), 2, D] (zero-filled;
    tq_kv_block_bounds fills them as rows arrive)."""
    return torch.zeros((cache.batch, cache.num_kv_heads, _block_count(cache.capacity, block_tokens), 2, cache.head_dim),
                       dtype=torch.float16, device=cache.buffer.device)


def _need_bounds(cache, bounds: torch.Tensor, block_tokens: int) -> None:
    _need(bounds, torch.float16, "bounds")
    if bounds.shape != (cache.batch, cache.num_kv_heads, _block_count(cache.capacity, block_tokens), 2, cache.head_dim):
        raise ValueError(f"bounds must be [B, Hkv, ceil(capacity / block_tokens), 2, D]; got {tuple(bounds.shape)}")


def _need_lens(t: torch.Tensor, batch: int, name: str) -> None:
    _need(t, torch.int32, name)
    if t.numel() != batch:
        raise ValueError(f"{name} must hold one entry per sequence; got {tuple(t.shape)}")


def tq_kv_block_bounds(cache, bounds: torch.Tensor, start: torch.Tensor, n_rows: int, block_tokens: int = 64,
                       status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Recompute the bounds of the blocks that rows [start[b], start[b] + n_rows) touch
    (after an append: its write_pos and n_new)."""
    _need_bounds(cache, bounds, block_tokens)
    _need_lens(start, cache.batch, "start")
    if status is not None:
        _need(status, torch.int32, "status")
    on = _on(stream, cache.buffer, bounds, start, status)
    _check("tq_kv_block_bounds", _fn(cache, "kv_block_bounds")(cache.ref(), int(block_tokens), start.data_ptr(), int(n_rows),
                                                              bounds.data_ptr(), status.data_ptr() if status is not None else None, on))
    return bounds


def sparse_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int, n_select: int,
                     block_tokens: int = 64, device="cuda") -> torch.Tensor:
    """A workspace for tq_select_blocks, tq_sdpa_blocks_decode and tq_sparse_decode of these sizes."""
    n = int(lib().tq_sparse_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, n_select, block_tokens))
    if n == 0:
        raise ValueError("invalid sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _need_blocks(cache, blocks: torch.Tensor) -> None:
    _need(blocks, torch.int32, "blocks")
    if blocks.dim() != 3 or blocks.shape[0] != cache.batch or blocks.shape[1] != cache.num_kv_heads:
        raise ValueError(f"blocks must be [B, Hkv, n_select]; got {tuple(blocks.shape)}")


def _need_query(cache, q: torch.Tensor, out: Optional[torch.Tensor], stream) -> torch.Tensor:
    _need(q, torch.float16, "q")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q.dtype, q.device, stream)
    _need(out, torch.float16, "out")
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cache.head_dim or out.shape != q.shape:
        raise ValueError(f"q must be [B, Hq, D]; got {tuple(q.shape)}")
    return out


def tq_select_blocks(bounds: torch.Tensor, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, workspace: torch.Tensor,
                     blocks: torch.Tensor, capacity: int, block_tokens: int = 64, n_first: int = 1, n_last: int = 1,
                     status: Optional[torch.Tensor] = None, stream=None, flags: int = 0) -> torch.Tensor:
    """The blocks [B, Hkv, n_select] that the query's score against the bounds of a cache of ``capacity`` tokens
    selects (ascending, -1 behind the last), written to ``blocks``."""
    _need(bounds, torch.float16, "bounds")
    _need(q, torch.float16, "q")
    _need(blocks, torch.int32, "blocks")
    _need(workspace, torch.uint8, "workspace")
    if status is not None:
        _need(status, torch.int32, "status")
    if q.dim() != 3 or blocks.dim() != 3 or bounds.dim() != 5 or blocks.shape[0] != q.shape[0]:
        raise ValueError("q must be [B, Hq, D], blocks [B, Hkv, n_select] and bounds [B, Hkv, n_blocks, 2, D]")
    b, hkv, n_select = blocks.shape
    if tuple(bounds.shape) != (b, hkv, _block_count(capacity, block_tokens), 2, q.shape[2]):
        raise ValueError(f"bounds do not match blocks, q and capacity; got {tuple(bounds.shape)}")
    _need_lens(seq_lens, b, "seq_lens")
    on = _on(stream, q, bounds, seq_lens, workspace, blocks, status)
    _check("tq_select_blocks", lib().tq_select_blocks(
        bounds.data_ptr(), q.data_ptr(), b, q.shape[1], hkv, q.shape[2], int(capacity), seq_lens.data_ptr(), int(max_seq_len),
        int(block_tokens), n_select, int(n_first), int(n_last), int(flags), workspace.data_ptr(), workspace.numel(),
        blocks.data_ptr(), status.data_ptr() if status is not None else None, on))
    return blocks


def tq_sdpa_blocks_decode(cache, q: torch.Tensor, blocks: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                          attn_scale: float, workspace: torch.Tensor, out: Optional[torch.Tensor] = None,
                          block_tokens: int = 64, status: Optional[torch.Tensor] = None, stream=None,
                          flags: int = 0) -> torch.Tensor:
    """Decode attention over the rows below seq_lens of the listed blocks [B, Hkv, n_select] (entries below 0: none)."""
    out = _need_query(cache, q, out, stream)
    _need_blocks(cache, blocks)
    _need_lens(seq_lens, cache.batch, "seq_lens")
    _need(workspace, torch.uint8, "workspace")
    if status is not None:
        _need(status, torch.int32, "status")
    on = _on(stream, cache.buffer, q, blocks, seq_lens, workspace, out, status)
    _check("tq_sdpa_blocks_decode", _fn(cache, "sdpa_blocks_decode")(
        cache.ref(), q.data_ptr(), q.shape[1], seq_lens.data_ptr(), int(max_seq_len), float(attn_scale), blocks.data_ptr(),
        blocks.shape[2], int(block_tokens), int(flags), workspace.data_ptr(), workspace.numel(), out.data_ptr(), status.data_ptr() if status is not None else None,
        on))
    return out


def tq_sparse_decode(cache, bounds: torch.Tensor, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                     attn_scale: float, workspace: torch.Tensor, blocks: torch.Tensor, out: Optional[torch.Tensor] = None,
                     block_tokens: int = 64, n_first: int = 1, n_last: int = 1, status: Optional[torch.Tensor] = None,
                     stream=None, flags: int = 0):
    """tq_select_blocks into ``blocks`` [B, Hkv, n_select], then tq_sdpa_blocks_decode over it; (out, blocks)."""
    out = _need_query(cache, q, out, stream)
    _need_bounds(cache, bounds, block_tokens)
    _need_blocks(cache, blocks)
    _need_lens(seq_lens, cache.batch, "seq_lens")
    _need(workspace, torch.uint8, "workspace")
    if status is not None:
        _need(status, torch.int32, "status")
    on = _on(stream, cache.buffer, bounds, q, blocks, seq_lens, workspace, out, status)
    _check("tq_sparse_decode", _fn(cache, "sparse_decode")(
        cache.ref(), bounds.data_ptr(), q.data_ptr(), q.shape[1], seq_lens.data_ptr(), int(max_seq_len), float(attn_scale),
        int(block_tokens), blocks.shape[2], int(n_first), int(n_last), int(flags), workspace.data_ptr(), workspace.numel(),
        blocks.data_ptr(), out.data_ptr(), status.data_ptr() if status is not None else None, on))
    return out, blocks


def weights_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
                      device="cuda") -> torch.Tensor:
    """A workspace for tq_sdpa_decode_weights of these sizes."""
    n = int(lib().tq_weights_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len))
    if n == 0:
        raise ValueError("invalid sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _need_weights(cache, t: torch.Tensor, name: str) -> None:
    _need(t, torch.float32, name)
    if t.shape != (cache.batch, cache.num_kv_heads, cache.capacity):
        raise ValueError(f"{name} must be [B, Hkv, capacity]; got {tuple(t.shape)}")


def tq_sdpa_decode_weights(cache, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, attn_scale: float,
                           weights: torch.Tensor, workspace: torch.Tensor, out: Optional[torch.Tensor] = None,
                           decay: float = 1.0, status: Optional[torch.Tensor] = None, stream=None,
                           flags: int = 0) -> torch.Tensor:
    """Fused decode attention that also sets weights[b, h, t] (fp32 [B, Hkv, capacity]) to decay times itself plus the
    attention weight of row t summed over the kv head's query heads, for t < seq_lens[b]."""
    out = _need_query(cache, q, out, stream)
    _need_weights(cache, weights, "weights")
    _need_lens(seq_lens, cache.batch, "seq_lens")
    _need(workspace, torch.uint8, "workspace")
    if status is not None:
        _need(status, torch.int32, "status")
    on = _on(stream, cache.buffer, q, seq_lens, weights, workspace, out, status)
    _check("tq_sdpa_decode_weights", _fn(cache, "sdpa_decode_weights")(
        cache.ref(), q.data_ptr(), q.shape[1], seq_lens.data_ptr(), int(max_seq_len), float(attn_scale), float(decay),
        weights.data_ptr(), int(flags), workspace.data_ptr(), workspace.numel(), out.data_ptr(), status.data_ptr() if status is not None else None, on))
    return out


def tq_kv_evict(src, dst, weights: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, keep: int, recent: int,
                dst_weights: torch.Tensor, dst_lens: torch.Tensor, kept: torch.Tensor,
                status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Move the last ``recent`` rows and the keep - recent others of greatest weight of every (sequence, kv head) of
    ``src`` to rows [0, keep) of ``dst`` (another cache of the same layout), with their weights; dst_lens int32 [B],
    kept int32 [B, Hkv, keep]: the src row of each dst row, -1 behind the last."""
    if getattr(src, "paged", False) != getattr(dst, "paged", False):
        raise ValueError("src and dst must both be contiguous or both be paged")
    _need_weights(src, weights, "weights")
    _need_weights(dst, dst_weights, "dst_weights")
    _need_lens(seq_lens, src.batch, "seq_lens")
    _need_lens(dst_lens, src.batch, "dst_lens")
    _need(kept, torch.int32, "kept")
    if kept.shape != (src.batch, src.num_kv_heads, int(keep)):
        raise ValueError(f"kept must be [B, Hkv, keep]; got {tuple(kept.shape)}")
    if status is not None:
        _need(status, torch.int32, "status")
    on = _on(stream, src.buffer, dst.buffer, weights, seq_lens, dst_weights, dst_lens, kept, status)
    _check("tq_kv_evict", _fn(src, "kv_evict")(
        src.ref(), dst.ref(), weights.data_ptr(), seq_lens.data_ptr(), int(max_seq_len), int(keep), int(recent), dst_weights.data_ptr(),
        dst_lens.data_ptr(), kept.data_ptr(), status.data_ptr() if status is not None else None, on))
