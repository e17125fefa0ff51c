"""Thin Python binding of libnd's C ABI (include/nd.h).

Argument marshalling only: shapes and dtypes are read from torch tensors, their
device pointers and the current CUDA stream are passed to the C entry points,
and a non-zero status raises NDError.  Every computation runs in the CUDA
kernels of libnd.so; there is no CPU or PyTorch fallback, and importing this
module on a machine without the built library raises.  torch is used for
device memory only (outputs and workspaces the caller did not supply).

Function names match the C ABI (nd_kv_append_quant, nd_swa_sink_decode, ...).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

ND_OK, ND_ERR_INVALID_ARG, ND_ERR_UNSUPPORTED, ND_ERR_CUDA, ND_ERR_WORKSPACE, ND_ERR_DEVICE = range(6)
ND_F32, ND_BF16 = 0, 1


class NDError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        name = _lib().nd_status_string(status).decode()
        extra = f" (cudaError {cuda_error})" if status == ND_ERR_CUDA else ""
        super().__init__(f"{fn} failed: {name}{extra}")


class _Cache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("sink_cap", ctypes.c_int), ("ring_cap", ctypes.c_int),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("sink_len", ctypes.c_void_p), ("ring_start", ctypes.c_void_p),
                ("ring_len", ctypes.c_void_p), ("seq_len", ctypes.c_void_p)]


class _CompressedCache(ctypes.Structure):
    _fields_ = [("kv", _Cache), ("k_sum", ctypes.c_void_p), ("v_sum", ctypes.c_void_p),
                ("block", ctypes.c_int), ("n_pinned", ctypes.c_int)]


class _ModelCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("d_model", "attn_dim", "num_heads", "num_kv_heads",
                                             "num_layers", "n_engram_sites", "max_seq_len",
                                             "kv_window")]


class _RopeCfg(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int),
                ("scaling", ctypes.c_int), ("theta", ctypes.c_float), ("factor", ctypes.c_float),
                ("low", ctypes.c_float), ("high", ctypes.c_float), ("orig_len", ctypes.c_float),
                ("magnitude", ctypes.c_float)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path) or _build._stale():
            path = _build.build()  # raises if the CUDA toolkit is missing
        lib = ctypes.CDLL(path)
        P, I, S, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
        F = ctypes.c_float
        sig = {
            "nd_version": (ctypes.c_char_p, []),
            "nd_status_string": (ctypes.c_char_p, [I]),
            "nd_last_cuda_error": (I, []),
            "nd_device_errors": (I, [P, I]),
            "nd_set_prefill_epilogue_wait_limit": (I, [ctypes.c_uint]),
            "nd_kv_append_quant": (I, [P, P, P, I, P]),
            "nd_kv_quant_rows": (I, [P, L, I, P, P, P]),
            "nd_kv_cache_from_prefill_workspace_size": (S, [I, I, I]),
            "nd_kv_cache_from_prefill": (I, [P, P, P, I, I, P, P, P, P, P, S, P]),
            "nd_swa_sink_decode_workspace_size": (S, [I, I, I, I, I]),
            "nd_swa_sink_decode": (I, [P, P, I, I, P, P, P, S, P]),
            "nd_swa_sink_decode_noalloc": (I, [P, P, I, I, P, P, P]),
            "nd_swa_sink_decode_step": (I, [P, P, P, P, I, I, P, P, P, S, P]),
            "nd_swa_sink_decode_step_host_workspace_size": (S, [I, I, I, I, I]),
            "nd_swa_sink_decode_step_host": (I, [P, P, P, P, I, I, P, P, P, S, P]),
            "nd_swa_sink_decode_step_host_packed": (I, [P, P, I, I, P, I, P, S, P]),
            "nd_compressed_decode_step_workspace_size": (S, [I, I, I, I, I]),
            "nd_compressed_decode_step": (I, [P, P, P, P, I, I, F, P, P, P, S, P]),
            "nd_swa_sink_prefill_workspace_size": (S, [I, I, I, I, I, I, F, I]),
            "nd_swa_sink_prefill": (I, [P, P, P, I, I, I, I, I, I, P, P, I, F, P, P, I, P, P, P, S, P]),
            "nd_swa_sink_prefill_tiles": (I, [P, I, I, I, I, I, F, I, P]),
            "nd_compressed_prefill_workspace_size": (S, [I, I, I, I, I, F, I]),
            "nd_compressed_prefill": (I, [P, P, P, I, I, I, I, I, I, I, I, F, P, P, P, S, P]),
            "nd_swa_sink_chunk_prefill_workspace_size": (S, [I, I, I, I, I, I, I, I]),
            "nd_swa_sink_chunk_prefill": (I, [P, P, P, I, P, I, I, P, P, P, S, P]),
            "nd_swa_sink_chunk_prefill_tiles": (I, [P, I, I, I, I, I, I, I, I, P]),
            "nd_kv_cache_read": (I, [P, I, I, I, P, P, P, P, P]),
            "nd_shared_prefix_decode_workspace_size": (S, [I, I, I, I, I, I]),
            "nd_shared_prefix_decode": (I, [P, P, P, I, I, P, P, P, S, P]),
            "nd_qk_norm_rope": (I, [P, P, I, I, I, I, I, I, L, L, P, P, F, F, P, P, P, P]),
            "nd_qk_norm_rope_append": (I, [P, P, P, P, I, L, L, L, P, P, F, F, P, I, P, P]),
            "nd_tree_layout": (I, [P, P, P, P, I, I, I, P, P, P, P]),
            "nd_tree_decode_workspace_size": (S, [I, I, I, I, I, I]),
            "nd_tree_decode": (I, [P, P, P, P, L, L, P, P, I, I, I, P, P, P, S, P]),
            "nd_tree_accept": (I, [P, P, P, P, P, I, I, I, P, P, P, P]),
            "nd_tree_commit": (I, [P, P, P, L, L, I, P, P, I, P]),
            "nd_rope_positions": (I, [P, P, I, I, I, I, I, I, L, L, P, P, P, P, P]),
            "nd_rope_apply": (I, [P, P, I, I, I, I, F, P]),
            "nd_kv_compress_pool": (I, [P, P, I, I, I, I, I, F, P, P, P]),
            "nd_kv_compress_pool_rope_workspace_size": (S, [I, I, F]),
            "nd_kv_compress_pool_rope": (I, [P, P, I, I, I, I, I, F, P, P, P, P, S, P]),
            "nd_kv_budget_window": (I, [P, P, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def library_path() -> str:
    _lib()
    return _build.LIB


EXPORTED = ("nd_version", "nd_status_string", "nd_last_cuda_error", "nd_device_errors",
            "nd_set_prefill_epilogue_wait_limit",
            "nd_kv_append_quant", "nd_kv_quant_rows", "nd_kv_cache_from_prefill_workspace_size", "nd_kv_cache_from_prefill", "nd_swa_sink_decode_workspace_size",
            "nd_swa_sink_decode", "nd_swa_sink_decode_noalloc", "nd_swa_sink_decode_step",
            "nd_swa_sink_decode_step_host_workspace_size", "nd_swa_sink_decode_step_host",
            "nd_swa_sink_decode_step_host_packed",
            "nd_compressed_decode_step_workspace_size", "nd_compressed_decode_step",
            "nd_swa_sink_prefill_workspace_size",
            "nd_swa_sink_prefill", "nd_swa_sink_prefill_tiles",
            "nd_compressed_prefill_workspace_size", "nd_compressed_prefill",
            "nd_swa_sink_chunk_prefill_workspace_size", "nd_swa_sink_chunk_prefill",
            "nd_swa_sink_chunk_prefill_tiles",
            "nd_kv_cache_read", "nd_shared_prefix_decode_workspace_size", "nd_shared_prefix_decode",
            "nd_tree_layout", "nd_tree_decode_workspace_size", "nd_tree_decode", "nd_tree_accept", "nd_tree_commit",
            "nd_qk_norm_rope", "nd_qk_norm_rope_append", "nd_rope_positions",
            "nd_rope_apply", "nd_kv_compress_pool", "nd_kv_compress_pool_rope_workspace_size",
            "nd_kv_compress_pool_rope", "nd_kv_budget_window")


def _check(fn: str, status: int):
    if status != ND_OK:
        raise NDError(fn, status, _lib().nd_last_cuda_error())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libnd takes CUDA tensors (device pointers)")
    if not t.is_contiguous():
        raise ValueError("libnd takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> int:
    # the current stream's handle alone: building the Stream object around it
    # takes longer than a small launch (2.8 us against 0.3 us on the GB300's CPU)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


# Tensors that a call makes belong to the stream it runs on: memory that the
# caching allocator gave out for another stream may still be in use there, and a
# workspace, which is let go when the call returns, would be handed to that
# stream's next tensor while the call's kernels are yet to run.

def _pool(stream):
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _pool(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t: torch.Tensor, stream, memory_format=torch.preserve_format) -> torch.Tensor:
    if stream is None:
        return torch.empty_like(t, memory_format=memory_format)
    with _pool(stream):
        return torch.empty_like(t, memory_format=memory_format)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    return _empty((max(nbytes, 16),), torch.uint8, device, stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return ND_F32
    if t.dtype == torch.bfloat16:
        return ND_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


# --------------------------------------------------------------------------
# Cache
# --------------------------------------------------------------------------

@dataclass
class KVCache:
    """Device tensors of one bounded cache in the nd_kv_cache layout."""
    k_codes: torch.Tensor   # int8 [B, Hkv, S+W, d]
    v_codes: torch.Tensor
    k_scale: torch.Tensor   # fp32 [B, Hkv, S+W, d/32]
    v_scale: torch.Tensor
    sink_len: torch.Tensor  # int32 [B]
    ring_start: torch.Tensor
    ring_len: torch.Tensor
    seq_len: torch.Tensor
    sink_cap: int
    ring_cap: int

    @classmethod
    def empty(cls, batch, n_kv_heads, head_dim, sink_cap, ring_cap, device="cuda"):
        ns = sink_cap + ring_cap
        z8 = lambda: torch.zeros((batch, n_kv_heads, ns, head_dim), dtype=torch.int8, device=device)
        zs = lambda: torch.zeros((batch, n_kv_heads, ns, head_dim // 32), dtype=torch.float32, device=device)
        zi = lambda: torch.zeros(batch, dtype=torch.int32, device=device)
        return cls(z8(), z8(), zs(), zs(), zi(), zi(), zi(), zi(), sink_cap, ring_cap)

    @property
    def batch(self):
        return self.k_codes.shape[0]

    @property
    def n_kv_heads(self):
        return self.k_codes.shape[1]

    @property
    def head_dim(self):
        return self.k_codes.shape[3]

    def struct(self) -> _Cache:
        return _Cache(self.batch, self.n_kv_heads, self.head_dim, self.sink_cap, self.ring_cap,
                      *(t.data_ptr() for t in (self.k_codes, self.v_codes, self.k_scale, self.v_scale,
                                               self.sink_len, self.ring_start, self.ring_len,
                                               self.seq_len)))

    def struct_ref(self):
        """A reference to the struct for ctypes, made again only when a tensor or a size changed (half the time)."""
        key = (self.k_codes.shape, self.sink_cap, self.ring_cap, self.k_codes.data_ptr(), self.v_codes.data_ptr(),
               self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.sink_len.data_ptr(),
               self.ring_start.data_ptr(), self.ring_len.data_ptr(), self.seq_len.data_ptr())
        kept = self.__dict__.get("_kept")
        if kept is None or kept[0] != key:
            self._check_layout()
            self._kept = kept = (key, ctypes.byref(self.struct()))
        return kept[1]

    def _check_layout(self):
        # the kernels go by the sizes: what is shorter would be read past its end
        codes = self.k_codes
        if codes.dim() != 4 or self.sink_cap < 0 or self.ring_cap < 0 or codes.shape[2] != self.sink_cap + self.ring_cap:
            raise ValueError("KVCache.k_codes must have shape [B, Hkv, sink_cap + ring_cap, d]")
        scales, rows = (*codes.shape[:3], codes.shape[3] // 32), codes.shape[:1]
        for name, shape, dtype in (("k_codes", codes.shape, torch.int8), ("v_codes", codes.shape, torch.int8),
                                   ("k_scale", scales, torch.float32), ("v_scale", scales, torch.float32),
                                   ("sink_len", rows, torch.int32), ("ring_start", rows, torch.int32),
                                   ("ring_len", rows, torch.int32), ("seq_len", rows, torch.int32)):
            t = getattr(self, name)
            if t.shape != shape or t.dtype != dtype or t.device != codes.device or not t.is_contiguous():
                raise ValueError(f"KVCache.{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                                 f"{codes.device}")

    def __getstate__(self):
        # copies and pickles take the fields alone: the kept reference is to this cache's struct, and cannot be pickled
        state = self.__dict__.copy()
        state.pop("_kept", None)
        return state


@dataclass
class CompressedCache:
    """A compressed-attention cache (nd_compressed_cache): kv's sink region
    holds n_pinned pinned tokens then the pooled blocks, its ring the exact
    window; k_sum / v_sum fp32 [B, Hkv, d] hold the open block's sums."""
    kv: KVCache
    k_sum: torch.Tensor
    v_sum: torch.Tensor
    block: int
    n_pinned: int = 0

    @classmethod
    def empty(cls, batch, n_kv_heads, head_dim, max_blocks, ring_cap, block, n_pinned=0, device="cuda"):
        kv = KVCache.empty(batch, n_kv_heads, head_dim, n_pinned + max_blocks, ring_cap, device)
        z = lambda: torch.zeros((batch, n_kv_heads, head_dim), dtype=torch.float32, device=device)
        return cls(kv, z(), z(), block, n_pinned)

    def struct(self) -> _CompressedCache:
        return _CompressedCache(self.kv.struct(), self.k_sum.data_ptr(), self.v_sum.data_ptr(), self.block,
                                self.n_pinned)


# --------------------------------------------------------------------------
# Entry points
# --------------------------------------------------------------------------

def nd_version() -> str:
    return _lib().nd_version().decode()


def nd_status_string(status: int) -> str:
    return _lib().nd_status_string(status).decode()


def nd_last_cuda_error() -> int:
    return int(_lib().nd_last_cuda_error())


def nd_device_errors(clear: bool = True) -> int:
    flags = ctypes.c_int(0)
    _check("nd_device_errors", _lib().nd_device_errors(ctypes.byref(flags), 1 if clear else 0))
    return flags.value


def nd_set_prefill_epilogue_wait_limit(polls: int) -> None:
    """Test hook: poll limit of the bf16 prefill's epilogue wait (0 = default)."""
    _check("nd_set_prefill_epilogue_wait_limit", _lib().nd_set_prefill_epilogue_wait_limit(int(polls)))


def nd_kv_append_quant(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                       to_sink: bool = False, stream=None) -> None:
    s = cache.struct()
    _check("nd_kv_append_quant", _lib().nd_kv_append_quant(
        ctypes.byref(s), _ptr(k_new), _ptr(v_new), 1 if to_sink else 0, _stream(stream)))


def nd_kv_quant_rows(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    _check("nd_kv_quant_rows", _lib().nd_kv_quant_rows(_ptr(x), n, d, _ptr(codes), _ptr(scales),
                                                       _stream(stream)))


def nd_kv_cache_from_prefill_workspace_size(cache_batch: int, sink_cap: int, ring_cap: int) -> int:
    return int(_lib().nd_kv_cache_from_prefill_workspace_size(cache_batch, sink_cap, ring_cap))


def nd_kv_cache_from_prefill(cache: KVCache, k: torch.Tensor, v: torch.Tensor, src_row: torch.Tensor,
                             seg_ids: Optional[torch.Tensor] = None, sink: Optional[torch.Tensor] = None,
                             src_seg: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> None:
    """Fill cache row e from segment src_seg[e] of batch row src_row[e] of a
    prefill's k / v (bf16 [B, T, Hkv, d]) as appending its tokens in order
    would; src_row / src_seg int32 [cache.batch] on the device."""
    B, T = k.shape[:2]
    if workspace is None:
        nbytes = nd_kv_cache_from_prefill_workspace_size(cache.batch, cache.sink_cap, cache.ring_cap)
        workspace = _scratch(nbytes, cache.k_codes.device, stream)
    s = cache.struct()
    _check("nd_kv_cache_from_prefill", _lib().nd_kv_cache_from_prefill(
        ctypes.byref(s), _ptr(k), _ptr(v), B, T, _ptr(seg_ids), _ptr(sink), _ptr(src_row), _ptr(src_seg),
        _ptr(workspace), workspace.numel(), _stream(stream)))


def nd_swa_sink_decode_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                      max_slots: int) -> int:
    return int(_lib().nd_swa_sink_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_slots))


def nd_swa_sink_decode(q: torch.Tensor, cache: KVCache, window: int, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    B, Hq, d = q.shape
    if out is None:
        out = _like(q, stream)
    if workspace is None:
        max_slots = cache.sink_cap + cache.ring_cap
        nbytes = nd_swa_sink_decode_workspace_size(B, Hq, cache.n_kv_heads, d, max_slots)
        workspace = _scratch(nbytes, q.device, stream)
    s = cache.struct()
    _check("nd_swa_sink_decode", _lib().nd_swa_sink_decode(
        _ptr(q), ctypes.byref(s), Hq, int(window), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return out


def nd_swa_sink_decode_step(q: torch.Tensor, cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                            window: int, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Ring-append the current token (k_new, v_new: bf16 [B][Hkv][d]) and
    attend with it: nd_kv_append_quant(to_sink=False) + nd_swa_sink_decode,
    in one launch when the sequence's CTAs fit a thread-block cluster."""
    B, Hq, d = q.shape
    if out is None:
        out = _like(q, stream)
    if workspace is None:
        nbytes = nd_swa_sink_decode_workspace_size(B, Hq, cache.n_kv_heads, d, cache.sink_cap + cache.ring_cap)
        workspace = _scratch(nbytes, q.device, stream)
    s = cache.struct()
    _check("nd_swa_sink_decode_step", _lib().nd_swa_sink_decode_step(
        _ptr(q), ctypes.byref(s), _ptr(k_new), _ptr(v_new), Hq, int(window), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def nd_swa_sink_decode_step_host_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                                max_slots: int) -> int:
    return int(_lib().nd_swa_sink_decode_step_host_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                                                  max_slots))


def nd_swa_sink_decode_step_host(q_host: torch.Tensor, cache: KVCache, k_new_host: torch.Tensor,
                                 v_new_host: torch.Tensor, window: int, out_host: torch.Tensor,
                                 lse_host: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                 stream=None, cache_struct=None) -> torch.Tensor:
    """nd_swa_sink_decode_step with q / k_new / v_new / out (/ lse) in host
    memory (CPU tensors, page-locked for asynchronous copies): the copies and
    the step are enqueued on the stream; out_host is valid once the stream
    has passed the call.  cache_struct: cache.struct(), built once by a
    caller that repeats the call on the same cache."""
    for t, name in ((q_host, "q_host"), (k_new_host, "k_new_host"), (v_new_host, "v_new_host"),
                    (out_host, "out_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    B, Hq, d = q_host.shape
    nk = cache.batch * cache.n_kv_heads * cache.head_dim
    if (B, d) != (cache.batch, cache.head_dim) or k_new_host.numel() != nk or v_new_host.numel() != nk or \
            out_host.numel() != q_host.numel() or (lse_host is not None and lse_host.numel() != B * Hq):
        raise ValueError("host buffer shapes do not match the cache")
    if workspace is None:
        nbytes = nd_swa_sink_decode_step_host_workspace_size(B, Hq, cache.n_kv_heads, d,
                                                             cache.sink_cap + cache.ring_cap)
        workspace = _scratch(nbytes, cache.k_codes.device, stream)
    s = cache_struct if cache_struct is not None else cache.struct()
    _check("nd_swa_sink_decode_step_host", _lib().nd_swa_sink_decode_step_host(
        q_host.data_ptr(), ctypes.byref(s), k_new_host.data_ptr(), v_new_host.data_ptr(), Hq, int(window),
        out_host.data_ptr(), None if lse_host is None else lse_host.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream(stream)))
    return out_host


def nd_swa_sink_decode_step_host_packed(in_host: torch.Tensor, cache: KVCache, n_q_heads: int, window: int,
                                        out_host: torch.Tensor, with_lse: bool = False,
                                        workspace: Optional[torch.Tensor] = None, stream=None,
                                        cache_struct=None) -> torch.Tensor:
    """nd_swa_sink_decode_step_host with packed host buffers: in_host one
    contiguous host tensor holding q | k_new | v_new (bf16, back to back),
    out_host one contiguous host tensor holding out (bf16) followed, with
    with_lse, by lse (fp32).  One copy each way.  Returns out_host."""
    s = cache_struct if cache_struct is not None else cache.struct()
    B, Hkv, d = s.batch, s.n_kv_heads, s.head_dim
    nin = (B * n_q_heads * d + 2 * B * Hkv * d) * 2
    nout = B * n_q_heads * d * 2 + (B * n_q_heads * 4 if with_lse else 0)
    # (this call sits on a per-token path: one cheap check per tensor)
    if in_host.is_cuda or not in_host.is_contiguous() or in_host.nbytes < nin:
        raise ValueError(f"in_host must be a contiguous host tensor of at least {nin} bytes")
    if out_host.is_cuda or not out_host.is_contiguous() or out_host.nbytes < nout:
        raise ValueError(f"out_host must be a contiguous host tensor of at least {nout} bytes")
    if workspace is None:
        nbytes = nd_swa_sink_decode_step_host_workspace_size(B, n_q_heads, Hkv, d, s.sink_cap + s.ring_cap)
        workspace = _scratch(nbytes, cache.k_codes.device, stream)
    _check("nd_swa_sink_decode_step_host_packed", _lib().nd_swa_sink_decode_step_host_packed(
        in_host.data_ptr(), ctypes.byref(s), n_q_heads, window, out_host.data_ptr(),
        1 if with_lse else 0, workspace.data_ptr(), workspace.nbytes, _stream(stream)))
    return out_host


NOALLOC_SCRATCH_BYTES = 512 << 10   # ND_NOALLOC_SCRATCH_BYTES in nd.h


def nd_swa_sink_decode_noalloc(q: torch.Tensor, cache: KVCache, window: int, out: torch.Tensor,
                               lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate device memory).  `out` must be given:
    this entry point allocates nothing.  Calls overlapping on the GPU race."""
    B, Hq, d = q.shape
    s = cache.struct()
    _check("nd_swa_sink_decode_noalloc", _lib().nd_swa_sink_decode_noalloc(
        _ptr(q), ctypes.byref(s), Hq, int(window), _ptr(out), _ptr(lse), _stream(stream)))
    return out


# The entry points below sit on a per-token path whose kernels take a few
# microseconds, about what a handful of attribute look-ups costs on the
# GB300's CPU: each tensor is looked at once, and addresses go to ctypes as
# plain integers.

def _here(t: torch.Tensor) -> int:
    """The index of t's device, which must be the current CUDA device (the
    library launches there)."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on {t.device}; libnd launches on the current CUDA device")
    return dev


def _on(stream, dev: int) -> int:
    """_stream() where the current device is known."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _addr(t: torch.Tensor, name: str, shape, dtype, dev: int) -> int:
    """The address of a contiguous tensor of this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _step(t: torch.Tensor, name: str) -> int:
    """The stride (elements) from one token to the next of [B, H, d] or
    [B, T, H, d] rows that may lie inside wider ones (a slice of a fused
    projection)."""
    if t.is_contiguous():
        return t.shape[-2] * t.shape[-1]
    shape, st = t.shape, t.stride()
    H, d = shape[-2:]
    step, ok = st[0], st[-1] == 1 and (st[-2] == d or H == 1)
    if len(shape) == 4:  # one stride for the tokens of all rows
        B, T = shape[:2]
        if T > 1:
            ok = ok and (B == 1 or step == T * st[1])
            step = st[1]
        B *= T
    else:
        B = shape[0]
    if not ok:
        raise ValueError(f"{name}: heads and channels must be contiguous, and the tokens evenly spaced")
    return step if B > 1 else H * d


def nd_kv_cache_read(cache: KVCache, window: int, dtype: torch.dtype = torch.bfloat16,
                     k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None, stream=None):
    """The cache's visible keys and values in position order: (k, v
    [B][rows][Hkv][d], positions int32 [B][rows], lengths int32 [B]), rows =
    sink_cap + min(ring_cap, window) unless k_out has more.  Rows from
    lengths[b] on keep what k_out / v_out held (nothing in particular when they
    are made here); their positions are -1."""
    codes = cache.k_codes
    dev = _here(codes)
    B, Hkv, _, d = codes.shape
    if k_out is None:
        if window < 1:
            raise ValueError("window must be at least 1")
        rows = cache.sink_cap + min(cache.ring_cap, window)
        shape = (B, rows, Hkv, d)
        k_out = _empty(shape, dtype, codes.device, stream)
        at_k = k_out.data_ptr()
    else:
        if k_out.dim() != 4:
            raise ValueError("k_out must have shape [B, rows, Hkv, d]")
        rows = k_out.shape[1]
        dtype = k_out.dtype
        shape = (B, rows, Hkv, d)
        at_k = _addr(k_out, "k_out", shape, dtype, dev)
    if v_out is None:
        v_out = _like(k_out, stream)
        at_v = v_out.data_ptr()
    else:
        at_v = _addr(v_out, "v_out", shape, dtype, dev)
    if positions is None:
        positions = _empty((B, rows), torch.int32, codes.device, stream)
        at_p = positions.data_ptr()
    else:
        at_p = _addr(positions, "positions", (B, rows), torch.int32, dev)
    if lengths is None:
        lengths = _like(cache.seq_len, stream)
        at_n = lengths.data_ptr()
    else:
        at_n = _addr(lengths, "lengths", (B,), torch.int32, dev)
    code = ND_BF16 if dtype == torch.bfloat16 else _dtype_code(k_out)
    _check("nd_kv_cache_read", _lib().nd_kv_cache_read(
        cache.struct_ref(), window, code, rows, at_k, at_v, at_p, at_n, _on(stream, dev)))
    return k_out, v_out, positions, lengths


def nd_shared_prefix_decode_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                           prefix_cap: int, max_slots: int) -> int:
    return int(_lib().nd_shared_prefix_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, prefix_cap,
                                                             max_slots))


def nd_shared_prefix_decode(q: torch.Tensor, prefix: KVCache, cache: KVCache, window: int,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """nd_swa_sink_decode for sequences that share the sink region of `prefix`
    (a cache of one row) in front of their own cache; returns out."""
    dev = _here(q)
    shape = q.shape
    B, Hq, d = shape
    k = cache.k_codes
    if k.shape[0] != B or k.shape[3] != d or k.get_device() != dev or prefix.k_codes.get_device() != dev:
        raise ValueError("q and the caches must agree on batch, head_dim and device")
    at_q = _addr(q, "q", shape, torch.bfloat16, dev)
    if out is None:
        out = _like(q, stream)
        at_out = out.data_ptr()
    else:
        at_out = _addr(out, "out", shape, torch.bfloat16, dev)
    if workspace is None:
        nbytes = nd_shared_prefix_decode_workspace_size(B, Hq, k.shape[1], d, prefix.sink_cap,
                                                        cache.sink_cap + cache.ring_cap)
        workspace = _scratch(nbytes, q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    _check("nd_shared_prefix_decode", _lib().nd_shared_prefix_decode(
        at_q, prefix.struct_ref(), cache.struct_ref(), Hq, window, at_out,
        None if lse is None else _addr(lse, "lse", (B, Hq), torch.float32, dev),
        workspace.data_ptr(), workspace.nbytes, _on(stream, dev)))
    return out


def _weight(w: Optional[torch.Tensor], name: str, d: int, dev: int) -> Optional[int]:
    return None if w is None else _addr(w, name, (d,), torch.float32, dev)


def _heads(t: Optional[torch.Tensor], out: Optional[torch.Tensor], name: str, B, T, d, dtype, dev: int, stream):
    """(heads, token stride, address, output's address, output) of q or k [B, T, heads, d]; None: no heads."""
    if t is None:
        return 0, 0, None, None, None
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != T or shape[3] != d or t.dtype != dtype or \
            t.get_device() != dev:
        raise ValueError(f"{name} must have shape [{B}, {T}, heads, {d}], q's type and device")
    step = _step(t, name)
    if out is None:
        out = _like(t, stream, torch.contiguous_format)
        return shape[2], step, t.data_ptr(), out.data_ptr(), out
    return shape[2], step, t.data_ptr(), _addr(out, name + "_out", shape, dtype, dev), out


def nd_qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                    k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, rope_theta: float = 0.0,
                    positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                    k_out: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of each head of q [B, T, Hq, d] and k [B, T, Hk, d] (bf16 or
    fp32; slices of a fused projection are taken as they are; either may be
    None) with weights fp32 [d], then the rotation at positions int32 [B, T]
    (None: t).  Returns (q_out, k_out), contiguous."""
    one = q if q is not None else k
    if one is None:
        raise ValueError("q or k must be given")
    dev = _here(one)
    B, T, _, d = one.shape
    dtype = one.dtype

    Hq, sq, pq, oq, q_out = _heads(q, q_out, "q", B, T, d, dtype, dev, stream)
    Hk, sk, pk, ok, k_out = _heads(k, k_out, "k", B, T, d, dtype, dev, stream)
    _check("nd_qk_norm_rope", _lib().nd_qk_norm_rope(
        pq, pk, _dtype_code(one), B, T, Hq, Hk, d, sq, sk, _weight(q_weight, "q_weight", d, dev),
        _weight(k_weight, "k_weight", d, dev), eps, rope_theta,
        None if positions is None else _addr(positions, "positions", (B, T), torch.int32, dev), oq, ok,
        _on(stream, dev)))
    return q_out, k_out


def nd_qk_norm_rope_append(q: torch.Tensor, cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                           q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, rope_theta: float = 0.0, pos_base: Optional[torch.Tensor] = None,
                           to_sink: bool = False, q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One decode token per sequence: q [B, Hq, d] and k_new [B, Hkv, d] (bf16,
    slices of a fused projection are taken as they are) are normalised per head
    and rotated at seq_len + pos_base (int32 tensor of one element, or None);
    k_new and v_new are quantised into the cache.  Returns q_out."""
    dev = _here(q)
    B, Hkv, _, d = cache.k_codes.shape
    shape, bf16 = q.shape, torch.bfloat16
    kv = (B, Hkv, d)
    if len(shape) != 3 or shape[0] != B or shape[2] != d or k_new.shape != kv or v_new.shape != kv or \
            q.dtype != bf16 or k_new.dtype != bf16 or v_new.dtype != bf16 or k_new.get_device() != dev or \
            v_new.get_device() != dev or cache.k_codes.get_device() != dev:
        raise ValueError(f"q, k_new and v_new must be bf16 [{B}, heads, {d}] (k_new, v_new: {Hkv} heads) on the "
                         "cache's device")
    if q_out is None:
        q_out = _like(q, stream, torch.contiguous_format)
        at_out = q_out.data_ptr()
    else:
        at_out = _addr(q_out, "q_out", shape, bf16, dev)
    base = None
    if pos_base is not None:
        if pos_base.numel() != 1 or pos_base.dtype != torch.int32 or pos_base.get_device() != dev:
            raise ValueError("pos_base must be one int32 on the cache's device")
        base = pos_base.data_ptr()
    _check("nd_qk_norm_rope_append", _lib().nd_qk_norm_rope_append(
        q.data_ptr(), cache.struct_ref(), k_new.data_ptr(), v_new.data_ptr(), shape[1], _step(q, "q"),
        _step(k_new, "k_new"), _step(v_new, "v_new"), _weight(q_weight, "q_weight", d, dev),
        _weight(k_weight, "k_weight", d, dev), eps, rope_theta, base, 1 if to_sink else 0,
        at_out, _on(stream, dev)))
    return q_out


TREE_MAX_NODES = 256                # ND_TREE_MAX_NODES in nd.h
ROPE_SCALINGS = {"none": 0, "linear": 1, "by_parts": 2}


@dataclass(frozen=True)
class RopeConfig:
    """How nd_rope_positions turns a head (nd_rope_cfg): its first rotary_dim
    channels (0: all), paired across halves or as neighbours, with the plain
    frequencies or scaled ones; inverse: the gradient's direction."""
    theta: float = 10000.0
    rotary_dim: int = 0
    interleaved: bool = False
    inverse: bool = False
    scaling: str = "none"            # "none", "linear" or "by_parts"
    factor: float = 1.0
    low: float = 1.0
    high: float = 32.0
    orig_len: float = 4096.0
    magnitude: float = 1.0

    def struct(self, head_dim: int) -> _RopeCfg:
        if self.scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        return _RopeCfg(self.rotary_dim or head_dim, int(self.interleaved), int(self.inverse), ROPE_SCALINGS[self.scaling],
                        self.theta, self.factor, self.low, self.high, self.orig_len, self.magnitude)

    def struct_ref(self, head_dim: int):
        """A reference to the struct for ctypes, made once per head_dim (the fields are frozen)."""
        kept = self.__dict__.get("_kept")
        if kept is None or kept[0] != head_dim:
            kept = (head_dim, ctypes.byref(self.struct(head_dim)))
            object.__setattr__(self, "_kept", kept)
        return kept[1]

    def __getstate__(self):
        state = self.__dict__.copy()  # (the kept reference cannot be pickled)
        state.pop("_kept", None)
        return state


def nd_rope_positions(q: Optional[torch.Tensor], k: Optional[torch.Tensor], rope: RopeConfig = RopeConfig(),
                      positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                      k_out: Optional[torch.Tensor] = None, stream=None):
    """The heads of q [B, T, Hq, d] and k [B, T, Hk, d] (bf16 or fp32; slices of
    a fused projection are taken as they are; either may be None) rotated at
    positions int32 [B, T] (None: t) as `rope` says.  Returns (q_out, k_out),
    contiguous.  For the gradient of the unrotated heads call it on the rotated
    heads' gradient with inverse=True."""
    one = q if q is not None else k
    if one is None:
        raise ValueError("q or k must be given")
    dev = _here(one)
    B, T, _, d = one.shape
    dtype = one.dtype
    Hq, sq, pq, oq, q_out = _heads(q, q_out, "q", B, T, d, dtype, dev, stream)
    Hk, sk, pk, ok, k_out = _heads(k, k_out, "k", B, T, d, dtype, dev, stream)
    _check("nd_rope_positions", _lib().nd_rope_positions(
        pq, pk, _dtype_code(one), B, T, Hq, Hk, d, sq, sk, rope.struct_ref(d),
        None if positions is None else _addr(positions, "positions", (B, T), torch.int32, dev), oq, ok,
        _on(stream, dev)))
    return q_out, k_out


def _ints(t: Optional[torch.Tensor], name: str, shape, dev: int) -> Optional[int]:
    return None if t is None else _addr(t, name, shape, torch.int32, dev)


def _parents(parents: torch.Tensor):
    dev = _here(parents)
    if parents.dim() != 2:
        raise ValueError("parents must have shape [B, n]")
    return dev, parents.shape[0], parents.shape[1], _addr(parents, "parents", parents.shape, torch.int32, dev)


def _one(t: Optional[torch.Tensor], name: str, dev: int) -> Optional[int]:
    if t is None:
        return None
    if t.numel() != 1 or t.dtype != torch.int32 or t.get_device() != dev:
        raise ValueError(f"{name} must be one int32 on cuda:{dev}")
    return t.data_ptr()


def _made(t: Optional[torch.Tensor], name: str, shape, dev: int, like: torch.Tensor, stream):
    """(tensor, address) of an int32 output, made here when it is not given."""
    if t is None:
        t = _empty(shape, torch.int32, like.device, stream)
        return t, t.data_ptr()
    return t, _addr(t, name, shape, torch.int32, dev)


def nd_tree_layout(parents: torch.Tensor, seq_len: Optional[torch.Tensor], window: int,
                   n_nodes: Optional[torch.Tensor] = None, pos_base: Optional[torch.Tensor] = None,
                   depth: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   mask: Optional[torch.Tensor] = None, stream=None):
    """Trees of drafted tokens from their parents (int32 [B, n], an earlier node
    or -1): (depth int32 [B, n], positions int32 [B, n] = seq_len + pos_base +
    depth, mask int32 [B, n, ceil(n/32)], the bits of the ancestors less than
    window above each node, itself among them).  Nodes from n_nodes[b] on are
    padding: depth and position -1, mask 0."""
    dev, B, n, at = _parents(parents)
    words = (n + 31) // 32
    depth, at_d = _made(depth, "depth", (B, n), dev, parents, stream)
    positions, at_p = _made(positions, "positions", (B, n), dev, parents, stream)
    mask, at_m = _made(mask, "mask", (B, n, words), dev, parents, stream)
    _check("nd_tree_layout", _lib().nd_tree_layout(
        at, _ints(n_nodes, "n_nodes", (B,), dev), _ints(seq_len, "seq_len", (B,), dev), _one(pos_base, "pos_base", dev),
        B, n, window, at_d, at_p, at_m, _on(stream, dev)))
    return depth, positions, mask


def nd_tree_accept(parents: torch.Tensor, tokens: torch.Tensor, target: torch.Tensor, max_path: int,
                   n_nodes: Optional[torch.Tensor] = None, root_target: Optional[torch.Tensor] = None,
                   path: Optional[torch.Tensor] = None, path_len: Optional[torch.Tensor] = None,
                   next: Optional[torch.Tensor] = None, stream=None):
    """The longest path of drafted tokens (int32 [B, n]) that the model's choices
    behind the nodes (target, int32 [B, n]) agree with: (path int32
    [B, max_path], -1 behind its end, path_len int32 [B], next int32 [B], the
    choice behind the path).  root_target: the choice behind the cache, which
    roots have to equal; None: roots hold."""
    dev, B, n, at = _parents(parents)
    if path is None and max_path < 1:
        raise ValueError("max_path must be at least 1")
    path, at_p = _made(path, "path", (B, max_path), dev, parents, stream)
    path_len, at_l = _made(path_len, "path_len", (B,), dev, parents, stream)
    next, at_n = _made(next, "next", (B,), dev, parents, stream)
    _check("nd_tree_accept", _lib().nd_tree_accept(
        at, _ints(n_nodes, "n_nodes", (B,), dev), _addr(tokens, "tokens", (B, n), torch.int32, dev),
        _addr(target, "target", (B, n), torch.int32, dev), _ints(root_target, "root_target", (B,), dev), B, n, max_path,
        at_p, at_l, at_n, _on(stream, dev)))
    return path, path_len, next


def _node_rows(k_new: torch.Tensor, v_new: torch.Tensor, cache: KVCache, dev: int):
    """n and the strides of the nodes' keys and values [B, n, Hkv, d]."""
    B, Hkv, _, d = cache.k_codes.shape
    shape = k_new.shape
    if len(shape) != 4 or shape[0] != B or shape[2] != Hkv or shape[3] != d or v_new.shape != shape or \
            k_new.dtype != torch.bfloat16 or v_new.dtype != torch.bfloat16 or k_new.get_device() != dev or \
            v_new.get_device() != dev or cache.k_codes.get_device() != dev:
        raise ValueError(f"k_new and v_new must be bf16 [{B}, n, {Hkv}, {d}] on the cache's device")
    return shape[1], _step(k_new, "k_new"), _step(v_new, "v_new")


def nd_tree_commit(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, path: torch.Tensor,
                   path_len: torch.Tensor, stream=None) -> None:
    """Append nodes path[b, :path_len[b]] (of k_new, v_new bf16 [B, n, Hkv, d])
    to each sequence's ring, as single appends in order would."""
    dev = _here(k_new)
    n, ks, vs = _node_rows(k_new, v_new, cache, dev)
    B = k_new.shape[0]
    if path.dim() != 2:
        raise ValueError("path must have shape [B, max_path]")
    m = path.shape[1]
    _check("nd_tree_commit", _lib().nd_tree_commit(
        cache.struct_ref(), k_new.data_ptr(), v_new.data_ptr(), ks, vs, n, _addr(path, "path", (B, m), torch.int32, dev),
        _addr(path_len, "path_len", (B,), torch.int32, dev), m, _on(stream, dev)))


def nd_tree_decode_workspace_size(batch: int, n: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                  max_slots: int) -> int:
    return int(_lib().nd_tree_decode_workspace_size(batch, n, n_q_heads, n_kv_heads, head_dim, max_slots))


def nd_tree_decode(q: torch.Tensor, cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, depth: torch.Tensor,
                   mask: torch.Tensor, window: int, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Attention of a tree's nodes (q bf16 [B, n, Hq, d]; k_new, v_new bf16
    [B, n, Hkv, d], slices of a fused projection are taken as they are) over the
    cache and the nodes that mask (nd_tree_layout's) names; returns out."""
    dev = _here(q)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must have shape [B, n, Hq, d]")
    n, ks, vs = _node_rows(k_new, v_new, cache, dev)
    B, _, Hq, d = shape
    if B != k_new.shape[0] or shape[1] != n or d != k_new.shape[3]:
        raise ValueError("q, k_new and v_new must agree on batch, nodes and head_dim")
    at_q = _addr(q, "q", shape, torch.bfloat16, dev)
    if out is None:
        out = _like(q, stream)
        at_out = out.data_ptr()
    else:
        at_out = _addr(out, "out", shape, torch.bfloat16, dev)
    if workspace is None:
        nbytes = nd_tree_decode_workspace_size(B, n, Hq, k_new.shape[2], d, cache.sink_cap + cache.ring_cap)
        workspace = _scratch(nbytes, q.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    _check("nd_tree_decode", _lib().nd_tree_decode(
        at_q, cache.struct_ref(), k_new.data_ptr(), v_new.data_ptr(), ks, vs,
        _addr(depth, "depth", (B, n), torch.int32, dev), _addr(mask, "mask", (B, n, (n + 31) // 32), torch.int32, dev), n,
        Hq, window, at_out, None if lse is None else _addr(lse, "lse", (B, Hq, n), torch.float32, dev),
        workspace.data_ptr(), workspace.nbytes, _on(stream, dev)))
    return out


def nd_compressed_decode_step_workspace_size(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                             max_slots: int) -> int:
    return int(_lib().nd_compressed_decode_step_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_slots))


def nd_compressed_decode_step(q: torch.Tensor, cache: CompressedCache, k_new: torch.Tensor, v_new: torch.Tensor,
                              window: int, rope_theta: float = 0.0, out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              stream=None, cache_struct=None) -> torch.Tensor:
    """Append the token at position seq_len (q, k_new, v_new before rotation)
    to the compressed cache and attend with it; returns out."""
    B, Hq, d = q.shape
    if out is None:
        out = _like(q, stream)
    kv = cache.kv
    if workspace is None:
        nbytes = nd_compressed_decode_step_workspace_size(B, Hq, kv.n_kv_heads, d, kv.sink_cap + kv.ring_cap)
        workspace = _scratch(nbytes, q.device, stream)
    s = cache_struct if cache_struct is not None else cache.struct()
    _check("nd_compressed_decode_step", _lib().nd_compressed_decode_step(
        _ptr(q), ctypes.byref(s), _ptr(k_new), _ptr(v_new), Hq, int(window), float(rope_theta), _ptr(out),
        _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def nd_swa_sink_prefill_workspace_size(dtype: int, batch: int, T: int, n_q_heads: int, n_kv_heads: int,
                                       head_dim: int, rope_theta: float = 0.0, block: int = 0) -> int:
    return int(_lib().nd_swa_sink_prefill_workspace_size(dtype, batch, T, n_q_heads, n_kv_heads, head_dim,
                                                         float(rope_theta), int(block)))


def nd_swa_sink_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        seg_ids: Optional[torch.Tensor] = None, sink: Optional[torch.Tensor] = None,
                        window: int = 0, rope_theta: float = 0.0,
                        pooled_k: Optional[torch.Tensor] = None, pooled_v: Optional[torch.Tensor] = None,
                        block: int = 0, out: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    dt = _dtype_code(q)
    if out is None:
        out = _like(q, stream)
    if workspace is None:
        nbytes = nd_swa_sink_prefill_workspace_size(dt, B, T, Hq, Hkv, d, rope_theta, block)
        workspace = _scratch(nbytes, q.device, stream)
    _check("nd_swa_sink_prefill", _lib().nd_swa_sink_prefill(
        _ptr(q), _ptr(k), _ptr(v), dt, B, T, Hq, Hkv, d, _ptr(seg_ids), _ptr(sink), int(window),
        float(rope_theta), _ptr(pooled_k), _ptr(pooled_v), int(block), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def nd_swa_sink_prefill_tiles(workspace: torch.Tensor, batch: int, T: int, n_q_heads: int, n_kv_heads: int,
                              head_dim: int, rope_theta: float = 0.0, block: int = 0) -> int:
    """128-row x 64-key tile products the bf16 prefill's attention kernel
    performed in its last call on `workspace` (reads the plan; synchronises)."""
    n = ctypes.c_longlong(0)
    _check("nd_swa_sink_prefill_tiles", _lib().nd_swa_sink_prefill_tiles(
        _ptr(workspace), batch, T, n_q_heads, n_kv_heads, head_dim, float(rope_theta), int(block), ctypes.byref(n)))
    return n.value


def nd_compressed_prefill_workspace_size(batch: int, T: int, n_q_heads: int, n_kv_heads: int, head_dim: int,
                                         rope_theta: float, block: int) -> int:
    return int(_lib().nd_compressed_prefill_workspace_size(batch, T, n_q_heads, n_kv_heads, head_dim,
                                                           float(rope_theta), int(block)))


def nd_compressed_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, block: int,
                          n_pinned: int = 0, rope_theta: float = 0.0, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Compressed attention with a pinned prefix of n_pinned exact keys (bf16
    q [B, T, Hq, d], k / v [B, T, Hkv, d] before rotation); returns out."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = _like(q, stream)
    if workspace is None:
        nbytes = nd_compressed_prefill_workspace_size(B, T, Hq, Hkv, d, rope_theta, block)
        workspace = _scratch(nbytes, q.device, stream)
    _check("nd_compressed_prefill", _lib().nd_compressed_prefill(
        _ptr(q), _ptr(k), _ptr(v), B, T, Hq, Hkv, d, int(window), int(block), int(n_pinned), float(rope_theta),
        _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def nd_swa_sink_chunk_prefill_workspace_size(batch: int, chunk: int, n_q_heads: int, n_kv_heads: int,
                                             head_dim: int, sink_cap: int, ring_cap: int, window: int) -> int:
    return int(_lib().nd_swa_sink_chunk_prefill_workspace_size(batch, chunk, n_q_heads, n_kv_heads, head_dim,
                                                               sink_cap, ring_cap, window))


def nd_swa_sink_chunk_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: KVCache, window: int,
                              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Prefill a chunk (q [B, Tc, Hq, d], k / v [B, Tc, Hkv, d], bf16, rotated)
    against the cache, then ring-append the chunk to it; returns out."""
    B, Tc, Hq, d = q.shape
    if out is None:
        out = _like(q, stream)
    if workspace is None:
        nbytes = nd_swa_sink_chunk_prefill_workspace_size(B, Tc, Hq, cache.n_kv_heads, d, cache.sink_cap,
                                                          cache.ring_cap, window)
        workspace = _scratch(nbytes, q.device, stream)
    s = cache.struct()
    _check("nd_swa_sink_chunk_prefill", _lib().nd_swa_sink_chunk_prefill(
        _ptr(q), _ptr(k), _ptr(v), Tc, ctypes.byref(s), Hq, int(window), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return out


def nd_swa_sink_chunk_prefill_tiles(workspace: torch.Tensor, batch: int, chunk: int, n_q_heads: int,
                                    n_kv_heads: int, head_dim: int, sink_cap: int, ring_cap: int,
                                    window: int) -> int:
    n = ctypes.c_longlong(0)
    _check("nd_swa_sink_chunk_prefill_tiles", _lib().nd_swa_sink_chunk_prefill_tiles(
        _ptr(workspace), batch, chunk, n_q_heads, n_kv_heads, head_dim, sink_cap, ring_cap, window, ctypes.byref(n)))
    return n.value


def nd_rope_apply(x: torch.Tensor, y: Optional[torch.Tensor] = None, rope_theta: float = 10000.0,
                  stream=None) -> torch.Tensor:
    B, T, H, d = x.shape
    if y is None:
        y = _like(x, stream)
    _check("nd_rope_apply", _lib().nd_rope_apply(_ptr(x), _ptr(y), B, T, H, d, float(rope_theta),
                                                 _stream(stream)))
    return y


def nd_kv_compress_pool(k: torch.Tensor, v: torch.Tensor, block: int, rope_theta: float = 0.0,
                        pooled_k: Optional[torch.Tensor] = None, pooled_v: Optional[torch.Tensor] = None,
                        stream=None):
    B, T, H, d = k.shape
    nb = T // block
    if pooled_k is None:
        pooled_k = _empty((B, nb, H, d), k.dtype, k.device, stream)
    if pooled_v is None:
        pooled_v = _empty((B, nb, H, d), v.dtype, v.device, stream)
    _check("nd_kv_compress_pool", _lib().nd_kv_compress_pool(
        _ptr(k), _ptr(v), B, T, H, d, int(block), float(rope_theta), _ptr(pooled_k), _ptr(pooled_v),
        _stream(stream)))
    return pooled_k, pooled_v


def nd_kv_compress_pool_rope_workspace_size(T: int, head_dim: int, rope_theta: float) -> int:
    return int(_lib().nd_kv_compress_pool_rope_workspace_size(T, head_dim, float(rope_theta)))


def nd_kv_compress_pool_rope(k: torch.Tensor, v: torch.Tensor, block: int, rope_theta: float = 0.0,
                             k_rot: Optional[torch.Tensor] = None, pooled_k: Optional[torch.Tensor] = None,
                             pooled_v: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None):
    """One pass over K and V: K rotated at every position (k_rot) and the
    pooled blocks (as nd_kv_compress_pool).  Returns (k_rot, pooled_k, pooled_v)."""
    B, T, H, d = k.shape
    nb = T // block
    if k_rot is None and rope_theta:
        k_rot = _like(k, stream)
    if pooled_k is None:
        pooled_k = _empty((B, nb, H, d), k.dtype, k.device, stream)
    if pooled_v is None:
        pooled_v = _empty((B, nb, H, d), v.dtype, v.device, stream)
    if workspace is None:
        workspace = _scratch(nd_kv_compress_pool_rope_workspace_size(T, d, rope_theta), k.device, stream)
    _check("nd_kv_compress_pool_rope", _lib().nd_kv_compress_pool_rope(
        _ptr(k), _ptr(v), B, T, H, d, int(block), float(rope_theta), _ptr(k_rot), _ptr(pooled_k), _ptr(pooled_v),
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return k_rot, pooled_k, pooled_v


def nd_kv_budget_window(d_model: int, attn_dim: int, num_heads: int, num_kv_heads: int, num_layers: int,
                        n_engram_sites: int, max_seq_len: int, kv_window: int = 0):
    """Returns (budget window, effective window)."""
    cfg = _ModelCfg(d_model, attn_dim or 0, num_heads, num_kv_heads, num_layers, n_engram_sites,
                    max_seq_len, kv_window or 0)
    b, e = ctypes.c_int(0), ctypes.c_int(0)
    _check("nd_kv_budget_window", _lib().nd_kv_budget_window(ctypes.byref(cfg), ctypes.byref(b),
                                                             ctypes.byref(e)))
    return b.value, e.value
