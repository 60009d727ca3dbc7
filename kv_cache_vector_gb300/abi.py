"""Thin ctypes binding of ``libtq.so`` (include/tq.h), same names as the C ABI.

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, turned into pointers, and the call is enqueued on torch's current
CUDA stream.  Every step of the codec and the attention runs in the library's
kernels.  There is no fallback: if ``libtq.so`` is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from contextlib import nullcontext
from dataclasses import dataclass
from functools import lru_cache

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtq.so")

TQ_F32, TQ_BF16 = 0, 1
STATUS = {0: "TQ_OK", 1: "TQ_ERR_INVALID_ARG", 2: "TQ_ERR_UNSUPPORTED", 3: "TQ_ERR_ALIGNMENT",
          4: "TQ_ERR_RANGE", 5: "TQ_ERR_WORKSPACE", 6: "TQ_ERR_CUDA", 7: "TQ_ERR_NOMEM"}

# every symbol include/tq.h declares
EXPORTS = ("tq_codebook_init", "tq_plan_create", "tq_plan_destroy", "tq_plan_signs",
           "tq_plan_codebook", "tq_encode", "tq_decode", "tq_append", "tq_attn_workspace_bytes", "tq_attn_paged_workspace_bytes",
           "tq_attn_decode", "tq_status_string", "tq_last_cuda_error", "tq_device_status",
           "tq_attn_decode_noalloc", "tq_attn_decode_ex", "tq_append_paged", "tq_attn_decode_paged",
           "tq_attn_decode_append_paged", "tq_plan_create_ex", "tq_plan_signs2", "tq_codebook_init_gaussian",
           "tq_attn_prefill_workspace_bytes", "tq_attn_prefill", "tq_qjl_matrix", "tq_encode_qjl",
           "tq_decode_qjl", "tq_attn_qjl_workspace_bytes", "tq_attn_decode_qjl",
           "tq_attn_prefill_paged_workspace_bytes", "tq_attn_prefill_paged",
           "tq_pages_workspace_bytes", "tq_pages_copy", "tq_pages_fork", "tq_pages_resize", "tq_pages_compact")


class TQError(RuntimeError):
    def __init__(self, fn: str, code: int, lib=None):
        self.code = code
        name = STATUS.get(code, str(code))
        extra = ""
        if code == 6 and lib is not None:
            extra = f" (cudaError {lib.tq_last_cuda_error()})"
        super().__init__(f"{fn} failed: {name}{extra}")


class CacheView(ctypes.Structure):
    _fields_ = [("k_packed", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("v_packed", ctypes.c_void_p), ("v_norm", ctypes.c_void_p),
                ("cap", ctypes.c_int64)]


class PagedCacheView(ctypes.Structure):
    _fields_ = [("k_packed", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("v_packed", ctypes.c_void_p), ("v_norm", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32)]


class PageTableView(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p)]


@lru_cache(maxsize=1)
def lib() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m kv_cache_vector_gb300.build` "
            "(needs nvcc); there is no CPU fallback")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float
    for name, res, args in [
        ("tq_codebook_init", i32, [i32, i32, vp, vp]),
        ("tq_plan_create", i32, [i32, u64, ctypes.POINTER(vp)]),
        ("tq_plan_create_ex", i32, [i32, u64, ctypes.c_uint32, ctypes.POINTER(vp)]),
        ("tq_plan_signs2", i32, [vp, vp]),
        ("tq_codebook_init_gaussian", i32, [i32, i32, vp, vp]),
        ("tq_plan_destroy", i32, [vp]),
        ("tq_plan_signs", i32, [vp, vp]),
        ("tq_plan_codebook", i32, [vp, i32, vp, vp]),
        ("tq_encode", i32, [vp, i32, vp, i32, i64, vp, vp, vp]),
        ("tq_decode", i32, [vp, i32, vp, vp, i64, vp, i32, vp]),
        ("tq_append", i32, [vp, i32, i32, vp, vp, i32, i32, i32, i64, CacheView, i64, vp]),
        ("tq_attn_workspace_bytes", ctypes.c_size_t, [i32, i32, i32, i32, i64]),
        ("tq_attn_paged_workspace_bytes", ctypes.c_size_t, [i32, i32, i32, i32, i64]),
        ("tq_attn_decode", i32, [vp, vp, i32, i32, i32, CacheView, i64, i32, i32, f32, f32, vp, vp,
                                 ctypes.c_size_t, vp]),
        ("tq_attn_decode_noalloc", i32, [vp, vp, i32, i32, i32, CacheView, i64, i32, i32, f32, f32,
                                         vp, vp]),
        ("tq_qjl_matrix", i32, [vp, vp, vp]),
        ("tq_encode_qjl", i32, [vp, i32, vp, vp, i32, i64, vp, vp, vp, vp]),
        ("tq_decode_qjl", i32, [vp, i32, vp, vp, vp, vp, i64, vp, i32, vp]),
        ("tq_attn_qjl_workspace_bytes", ctypes.c_size_t, [i32, i32, i32, i32, i64]),
        ("tq_attn_decode_qjl", i32, [vp, vp, vp, i32, i32, i32, CacheView, vp, i64, i32, i32, f32, vp, vp,
                                     ctypes.c_size_t, vp]),
        ("tq_attn_decode_ex", i32, [vp, vp, i32, i32, i32, CacheView, i64, i32, i32, f32, f32, vp, vp, vp,
                                    ctypes.c_size_t, vp]),
        ("tq_append_paged", i32, [vp, i32, i32, vp, vp, i32, i32, i32, PagedCacheView, vp, i32, vp, vp]),
        ("tq_attn_decode_paged", i32, [vp, vp, i32, i32, i32, PagedCacheView, vp, i32, vp, i64, i32, i32,
                                       f32, f32, vp, vp, ctypes.c_size_t, vp]),
        ("tq_attn_decode_append_paged", i32, [vp, vp, vp, vp, i32, i32, i32, i32, PagedCacheView, vp, i32, vp,
                                              i64, i32, i32, f32, f32, vp, vp, ctypes.c_size_t, vp]),
        ("tq_attn_prefill_workspace_bytes", ctypes.c_size_t, [i32, i32, i32, i32, i64, i32]),
        ("tq_attn_prefill", i32, [vp, vp, i32, i32, i32, i32, CacheView, vp, i32, i32, f32, vp, vp,
                                  ctypes.c_size_t, vp]),
        ("tq_attn_prefill_paged_workspace_bytes", ctypes.c_size_t, [i32, i32, i32]),
        ("tq_attn_prefill_paged", i32, [vp, vp, i64, i32, i32, i32, PagedCacheView, vp, i32, vp, vp, i32, i32, i32,
                                        f32, vp, i32, vp, ctypes.c_size_t, vp]),
        ("tq_pages_workspace_bytes", ctypes.c_size_t, [i32, i32, i64]),
        ("tq_pages_copy", i32, [vp, vp, i32, i32, i32, i32, i32, vp, vp, i64, vp, ctypes.c_size_t, vp]),
        ("tq_pages_fork", i32, [PageTableView, vp, PageTableView, i32, i32, vp, i32, i32, i32, i32, i32, vp, vp,
                                ctypes.c_size_t, vp]),
        ("tq_pages_resize", i32, [PageTableView, vp, PageTableView, i32, i32, vp, i32, i32, i32, i32, i32, vp, vp,
                                  ctypes.c_size_t, vp]),
        ("tq_pages_compact", i32, [PageTableView, PageTableView, vp, i32, i32, vp, i32, i32, i32, i32, i32, vp, vp,
                                   ctypes.c_size_t, vp]),
        ("tq_status_string", ctypes.c_char_p, [i32]),
        ("tq_last_cuda_error", i32, []),
        ("tq_device_status", i32, [i32, ctypes.POINTER(i32)]),
    ]:
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def _check(fn: str, code: int):
    if code != 0:
        raise TQError(fn, code, lib())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    raise TypeError(f"dtype {t.dtype} not supported (fp32 or bf16)")


def _cuda(*ts):
    for t in ts:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
            raise ValueError("expected contiguous CUDA tensors")


def tq_codebook_init(d: int, bits: int):
    """Lloyd-Max codebook (double): (centroids[2^b], boundaries[2^b - 1])."""
    c = np.empty(1 << bits, np.float64)
    b = np.empty((1 << bits) - 1, np.float64)
    _check("tq_codebook_init", lib().tq_codebook_init(d, bits, c.ctypes.data, b.ctypes.data))
    return c, b


PLAN_GAUSSIAN_CODEBOOK = 1  # TQ_PLAN_GAUSSIAN_CODEBOOK
PLAN_TWO_SIDED_SIGNS = 2    # TQ_PLAN_TWO_SIDED_SIGNS


class Plan:
    """Owns a tq_plan (host object: d, seed, format flags, signs, fp32 codebooks)."""

    def __init__(self, d: int, seed: int, flags: int = 0):
        h = ctypes.c_void_p()
        _check("tq_plan_create_ex", lib().tq_plan_create_ex(d, ctypes.c_uint64(seed), flags, ctypes.byref(h)))
        self.handle, self.d, self.seed, self.flags = h, d, seed, flags

    def signs(self) -> np.ndarray:
        s = np.empty(self.d, np.int8)
        _check("tq_plan_signs", lib().tq_plan_signs(self.handle, s.ctypes.data))
        return s

    def signs2(self) -> np.ndarray:
        s = np.empty(self.d, np.int8)
        _check("tq_plan_signs2", lib().tq_plan_signs2(self.handle, s.ctypes.data))
        return s

    def codebook(self, bits: int):
        c = np.empty(1 << bits, np.float32)
        b = np.empty((1 << bits) - 1, np.float32)
        _check("tq_plan_codebook", lib().tq_plan_codebook(self.handle, bits, c.ctypes.data, b.ctypes.data))
        return c, b

    def close(self):
        if getattr(self, "handle", None):
            lib().tq_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tq_plan_create(d: int, seed: int, flags: int = 0) -> Plan:
    return Plan(d, seed, flags)


def tq_codebook_init_gaussian(d: int, bits: int):
    """(centroids[2^b], boundaries[2^b - 1]) of N(0, 1/d), float64, on the host."""
    c = np.empty(1 << bits, np.float64)
    b = np.empty((1 << bits) - 1, np.float64)
    _check("tq_codebook_init_gaussian", lib().tq_codebook_init_gaussian(d, bits, c.ctypes.data, b.ctypes.data))
    return c, b


def tq_encode(plan: Plan, bits: int, x: torch.Tensor, packed: torch.Tensor | None = None,
              norms: torch.Tensor | None = None):
    """x: [n, d] fp32/bf16 CUDA -> (packed [n, d*bits/8] uint8, norms [n] fp32)."""
    x2 = x.reshape(-1, plan.d)
    n = x2.shape[0]
    if packed is None:
        packed = torch.empty(n, plan.d * bits // 8, dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty(n, dtype=torch.float32, device=x.device)
    _cuda(x2, packed, norms)
    _check("tq_encode", lib().tq_encode(plan.handle, bits, x2.data_ptr(), _dt(x2), n,
                                        packed.data_ptr(), norms.data_ptr(), _stream(x2)))
    return packed, norms


def tq_decode(plan: Plan, bits: int, packed: torch.Tensor, norms: torch.Tensor,
              out_dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    n = norms.numel()
    if out is None:
        out = torch.empty(n, plan.d, dtype=out_dtype, device=packed.device)
    _cuda(packed, norms, out)
    _check("tq_decode", lib().tq_decode(plan.handle, bits, packed.data_ptr(), norms.data_ptr(), n,
                                        out.data_ptr(), _dt(out), _stream(out)))
    return out


@dataclass
class Cache:
    """One layer of a packed KV cache (caller-owned device tensors)."""
    k_packed: torch.Tensor  # [B, Hkv, cap, d*kb/8] uint8
    k_norm: torch.Tensor    # [B, Hkv, cap] fp32
    v_packed: torch.Tensor  # [B, Hkv, cap, d*vb/8] uint8
    v_norm: torch.Tensor    # [B, Hkv, cap] fp32
    k_bits: int
    v_bits: int

    @staticmethod
    def empty(B, Hkv, cap, d, k_bits, v_bits, device="cuda"):
        return Cache(torch.zeros(B, Hkv, cap, d * k_bits // 8, dtype=torch.uint8, device=device),
                     torch.zeros(B, Hkv, cap, dtype=torch.float32, device=device),
                     torch.zeros(B, Hkv, cap, d * v_bits // 8, dtype=torch.uint8, device=device),
                     torch.zeros(B, Hkv, cap, dtype=torch.float32, device=device), k_bits, v_bits)

    @property
    def cap(self) -> int:
        return self.k_norm.shape[2]

    def view(self) -> CacheView:
        _cuda(self.k_packed, self.k_norm, self.v_packed, self.v_norm)
        return CacheView(self.k_packed.data_ptr(), self.k_norm.data_ptr(), self.v_packed.data_ptr(),
                         self.v_norm.data_ptr(), self.cap)


def tq_append(plan: Plan, cache: Cache, k_new: torch.Tensor, v_new: torch.Tensor, pos: int):
    """k_new, v_new: [B, Hkv, n_new, d] fp32/bf16 -> written at positions pos..pos+n_new-1."""
    B, Hkv, n_new, d = k_new.shape
    if v_new.shape != k_new.shape or v_new.dtype != k_new.dtype or d != plan.d:
        raise ValueError("k_new / v_new must both be [B, Hkv, n_new, d] of one dtype")
    _cuda(k_new, v_new)
    _check("tq_append", lib().tq_append(plan.handle, cache.k_bits, cache.v_bits, k_new.data_ptr(),
                                        v_new.data_ptr(), _dt(k_new), B, Hkv, n_new, cache.view(),
                                        pos, _stream(k_new)))


def tq_attn_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, ctx_len: int) -> int:
    return int(lib().tq_attn_workspace_bytes(B, Hq, Hkv, d, ctx_len))


def tq_attn_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_ctx: int) -> int:
    return int(lib().tq_attn_paged_workspace_bytes(B, Hq, Hkv, d, max_ctx))


def tq_attn_decode(plan: Plan, q: torch.Tensor, cache: Cache, ctx_len: int, scale: float,
                   sparse_v_threshold: float = 0.0, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """q: [B, Hq, d] bf16 -> out [B, Hq, d] fp32."""
    B, Hq, d = q.shape
    Hkv = cache.k_norm.shape[1]
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    need = tq_attn_workspace_bytes(B, Hq, Hkv, d, ctx_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(q, out, workspace)
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    _check("tq_attn_decode", lib().tq_attn_decode(
        plan.handle, q.data_ptr(), B, Hq, Hkv, cache.view(), ctx_len, cache.k_bits, cache.v_bits,
        ctypes.c_float(scale), ctypes.c_float(sparse_v_threshold), out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(q)))
    return out


def tq_attn_decode_ex(plan: Plan, q: torch.Tensor, cache: Cache, ctx_len: int, scale: float,
                      sparse_v_threshold: float = 0.0, out: torch.Tensor | None = None,
                      v_rows_read: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None):
    """tq_attn_decode that also returns, per (batch, KV head), how many cached
    rows' V bytes the call read: (out [B, Hq, d] fp32, v_rows_read [B, Hkv] int32)."""
    B, Hq, d = q.shape
    Hkv = cache.k_norm.shape[1]
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    if v_rows_read is None:
        v_rows_read = torch.empty(B, Hkv, dtype=torch.int32, device=q.device)
    need = tq_attn_workspace_bytes(B, Hq, Hkv, d, ctx_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(q, out, workspace, v_rows_read)
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    _i32(v_rows_read, "v_rows_read")
    _check("tq_attn_decode_ex", lib().tq_attn_decode_ex(
        plan.handle, q.data_ptr(), B, Hq, Hkv, cache.view(), ctx_len, cache.k_bits, cache.v_bits,
        ctypes.c_float(scale), ctypes.c_float(sparse_v_threshold), out.data_ptr(), v_rows_read.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(q)))
    return out, v_rows_read


def tq_attn_decode_noalloc(plan: Plan, q: torch.Tensor, cache: Cache, ctx_len: int, scale: float,
                           sparse_v_threshold: float = 0.0,
                           out: torch.Tensor | None = None) -> torch.Tensor:
    """As tq_attn_decode, without a workspace: for callers that may not
    allocate device memory while they run.  The library's fixed 8 MiB device
    array holds the split-K partials; sizes that need more raise TQError
    (TQ_ERR_WORKSPACE).  Calls that overlap on the GPU share that array and
    race.  (This wrapper allocates `out` only when none is passed.)"""
    B, Hq, d = q.shape
    Hkv = cache.k_norm.shape[1]
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    _cuda(q, out)
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    _check("tq_attn_decode_noalloc", lib().tq_attn_decode_noalloc(
        plan.handle, q.data_ptr(), B, Hq, Hkv, cache.view(), ctx_len, cache.k_bits, cache.v_bits,
        ctypes.c_float(scale), ctypes.c_float(sparse_v_threshold), out.data_ptr(), _stream(q)))
    return out


@dataclass
class PagedCache:
    """One layer of a paged KV cache (caller-owned device tensors): pages of
    page_size positions, each holding every KV head."""
    k_packed: torch.Tensor  # [n_pages, Hkv, page_size, d*kb/8] uint8
    k_norm: torch.Tensor    # [n_pages, Hkv, page_size] fp32
    v_packed: torch.Tensor  # [n_pages, Hkv, page_size, d*vb/8] uint8
    v_norm: torch.Tensor    # [n_pages, Hkv, page_size] fp32
    k_bits: int
    v_bits: int

    @staticmethod
    def empty(n_pages, Hkv, page_size, d, k_bits, v_bits, device="cuda"):
        return PagedCache(
            torch.zeros(n_pages, Hkv, page_size, d * k_bits // 8, dtype=torch.uint8, device=device),
            torch.zeros(n_pages, Hkv, page_size, dtype=torch.float32, device=device),
            torch.zeros(n_pages, Hkv, page_size, d * v_bits // 8, dtype=torch.uint8, device=device),
            torch.zeros(n_pages, Hkv, page_size, dtype=torch.float32, device=device), k_bits, v_bits)

    @property
    def n_pages(self) -> int:
        return self.k_norm.shape[0]

    @property
    def Hkv(self) -> int:
        return self.k_norm.shape[1]

    @property
    def page_size(self) -> int:
        return self.k_norm.shape[2]

    def view(self) -> PagedCacheView:
        _cuda(self.k_packed, self.k_norm, self.v_packed, self.v_norm)
        return PagedCacheView(self.k_packed.data_ptr(), self.k_norm.data_ptr(), self.v_packed.data_ptr(),
                              self.v_norm.data_ptr(), self.n_pages, self.page_size)


def _i32(t: torch.Tensor, name: str):
    _cuda(t)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")


def tq_append_paged(plan: Plan, cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor,
                    block_table: torch.Tensor, positions: torch.Tensor):
    """k_new, v_new: [B, Hkv, d] fp32/bf16; block_table [B, max_pages] int32;
    positions [B] int32: row (b, h) goes to position positions[b] of sequence b."""
    B, Hkv, d = k_new.shape
    if v_new.shape != k_new.shape or v_new.dtype != k_new.dtype or d != plan.d or Hkv != cache.Hkv:
        raise ValueError("k_new / v_new must both be [B, Hkv, d] of one dtype")
    _cuda(k_new, v_new)
    _i32(block_table, "block_table")
    _i32(positions, "positions")
    _check("tq_append_paged", lib().tq_append_paged(
        plan.handle, cache.k_bits, cache.v_bits, k_new.data_ptr(), v_new.data_ptr(), _dt(k_new), B, Hkv,
        cache.view(), block_table.data_ptr(), block_table.shape[1], positions.data_ptr(), _stream(k_new)))


def tq_attn_decode_paged(plan: Plan, q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor,
                         ctx_lens: torch.Tensor, max_ctx: int, scale: float,
                         sparse_v_threshold: float = 0.0, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None) -> torch.Tensor:
    """q: [B, Hq, d] bf16; block_table [B, max_pages] int32; ctx_lens [B] int32
    (each at most max_ctx) -> out [B, Hq, d] fp32."""
    B, Hq, d = q.shape
    Hkv = cache.Hkv
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    need = tq_attn_paged_workspace_bytes(B, Hq, Hkv, d, max_ctx)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(q, out, workspace)
    _i32(block_table, "block_table")
    _i32(ctx_lens, "ctx_lens")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    _check("tq_attn_decode_paged", lib().tq_attn_decode_paged(
        plan.handle, q.data_ptr(), B, Hq, Hkv, cache.view(), block_table.data_ptr(), block_table.shape[1],
        ctx_lens.data_ptr(), max_ctx, cache.k_bits, cache.v_bits, ctypes.c_float(scale),
        ctypes.c_float(sparse_v_threshold), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream(q)))
    return out


def tq_attn_decode_append_paged(plan: Plan, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                cache: PagedCache, block_table: torch.Tensor, positions: torch.Tensor,
                                max_ctx: int, scale: float, sparse_v_threshold: float = 0.0,
                                out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """One decode step: append k_new/v_new [B, Hkv, d] (fp32 or bf16) at
    positions [B] int32, then attend q [B, Hq, d] bf16 over positions + 1
    (at most max_ctx) -> out [B, Hq, d] fp32."""
    B, Hq, d = q.shape
    Hkv = cache.Hkv
    if tuple(k_new.shape) != (B, Hkv, d) or tuple(v_new.shape) != (B, Hkv, d):
        raise ValueError("k_new and v_new must be [B, Hkv, d]")
    if k_new.dtype != v_new.dtype:
        raise TypeError("k_new and v_new must share a dtype")
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    need = tq_attn_paged_workspace_bytes(B, Hq, Hkv, d, max_ctx)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(q, k_new, v_new, out, workspace)
    _i32(block_table, "block_table")
    _i32(positions, "positions")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    k_new, v_new = k_new.contiguous(), v_new.contiguous()
    _check("tq_attn_decode_append_paged", lib().tq_attn_decode_append_paged(
        plan.handle, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), _dt(k_new), B, Hq, Hkv, cache.view(),
        block_table.data_ptr(), block_table.shape[1], positions.data_ptr(), max_ctx, cache.k_bits,
        cache.v_bits, ctypes.c_float(scale), ctypes.c_float(sparse_v_threshold), out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(q)))
    return out


def tq_attn_prefill(plan: Plan, q: torch.Tensor, cache: Cache, q_start: torch.Tensor, scale: float,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """q: [B, T, Hq, d] bf16; q_start [B] int32 (token t of sequence b sits at
    q_start[b] + t and attends causally) -> out [B, T, Hq, d] fp32."""
    B, T, Hq, d = q.shape
    Hkv = cache.k_norm.shape[1]
    if out is None:
        out = torch.empty(B, T, Hq, d, dtype=torch.float32, device=q.device)
    need = int(lib().tq_attn_prefill_workspace_bytes(B, T, Hq, Hkv, cache.cap, d))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(q, out, workspace)
    _i32(q_start, "q_start")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    _check("tq_attn_prefill", lib().tq_attn_prefill(
        plan.handle, q.contiguous().data_ptr(), B, T, Hq, Hkv, cache.view(), q_start.data_ptr(), cache.k_bits,
        cache.v_bits, ctypes.c_float(scale), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream(q)))
    return out


def tq_attn_prefill_paged_workspace_bytes(Hq: int, Hkv: int, d: int) -> int:
    return int(lib().tq_attn_prefill_paged_workspace_bytes(Hq, Hkv, d))


def tq_attn_prefill_paged(plan: Plan, q: torch.Tensor, cu_q: torch.Tensor, cache: PagedCache,
                          block_table: torch.Tensor, ctx_lens: torch.Tensor, scale: float, window: int = 0,
                          out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """q: [n_q, Hq, d] bf16, the query tokens of all sequences one after the
    other; cu_q [B + 1] int32: sequence b's are rows cu_q[b] .. cu_q[b + 1] - 1
    and sit at the end of its ctx_lens[b] positions, each attending causally
    (over the last `window` positions, 0: all) -> out [n_q, Hq, d] bf16 or
    fp32.  Rows outside every sequence keep what `out` held (zeros if none is
    passed)."""
    n_q, Hq, d = q.shape
    B = ctx_lens.numel()
    rows = cache.k_norm.shape
    if d != plan.d or len(rows) != 3 or cache.v_norm.shape != rows or \
            cache.k_packed.shape != (*rows, d * cache.k_bits // 8) or \
            cache.v_packed.shape != (*rows, d * cache.v_bits // 8):
        raise ValueError("q and the cache's arrays must have the plan's head dimension and one geometry")
    if cu_q.numel() != B + 1 or block_table.shape[0] != B:
        raise ValueError("cu_q [B + 1], ctx_lens [B] and block_table [B, max_pages] expected")
    if not 0 <= window < 2 ** 31:
        raise ValueError("window must be in [0, 2^31)")
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    if (cache.k_packed.dtype, cache.v_packed.dtype, cache.k_norm.dtype, cache.v_norm.dtype) != \
            (torch.uint8, torch.uint8, torch.float32, torch.float32):
        raise TypeError("packed rows must be uint8 and norms fp32")
    _cuda(q)
    dev = q.device
    _ints(dev, cu_q, block_table, ctx_lens)
    _same_device(dev, cache.k_packed, cache.k_norm, cache.v_packed, cache.v_norm)
    with _on(dev):
        if out is None:
            out = torch.zeros(n_q, Hq, d, dtype=out_dtype, device=dev)
        _cuda(out)
        _same_device(dev, out)
        if out.shape != q.shape:
            raise ValueError("out must be [n_q, Hq, d]")
        ws = _scratch(workspace, dev, tq_attn_prefill_paged_workspace_bytes, Hq, cache.Hkv, d)
        _check("tq_attn_prefill_paged", lib().tq_attn_prefill_paged(
            plan.handle, q.data_ptr(), n_q, B, Hq, cache.Hkv, cache.view(), block_table.data_ptr(),
            block_table.shape[1], cu_q.data_ptr(), ctx_lens.data_ptr(), window, cache.k_bits, cache.v_bits,
            scale, out.data_ptr(), _dt(out), ws.data_ptr(), ws.nbytes, _raw_stream(dev)))
    return out


# ------------------------------------------------------------ upkeep of the pages

class PagedLayers:
    """The layers of one pool: paged caches of one geometry that share a block
    table.  Holds their tensors with the addresses, so that a call passes them
    as they are; a cache that is given other tensors needs new PagedLayers."""

    def __init__(self, layers):
        layers = [layers] if isinstance(layers, PagedCache) else list(layers)
        if not layers:
            raise ValueError("at least one layer")
        c = layers[0]
        for x in layers:
            for t in (x.k_packed, x.k_norm, x.v_packed, x.v_norm):
                _cuda(t)
                if t.device != c.k_norm.device:
                    raise ValueError("the layers must be on one device")
            if (x.k_packed.dtype, x.v_packed.dtype) != (torch.uint8,) * 2 or \
                    (x.k_norm.dtype, x.v_norm.dtype) != (torch.float32,) * 2:
                raise TypeError("packed rows must be uint8 and norms fp32")
            if (x.k_packed.shape, x.v_packed.shape, x.k_norm.shape, x.v_norm.shape, x.k_bits, x.v_bits) != \
                    (c.k_packed.shape, c.v_packed.shape, c.k_norm.shape, c.k_norm.shape, c.k_bits, c.v_bits):
                raise ValueError("the layers must have one geometry")
        self.layers = layers
        # the tensors themselves: a PagedCache may be given others
        self._tensors = [(x.k_packed, x.k_norm, x.v_packed, x.v_norm) for x in layers]
        self.k_bits, self.v_bits, self.device = c.k_bits, c.v_bits, c.k_norm.device
        self.n_pages, self.Hkv, self.page_size = c.k_norm.shape
        self.d = c.k_packed.shape[-1] * 8 // c.k_bits
        if tuple(c.k_packed.shape) != (*c.k_norm.shape, self.d * c.k_bits // 8) or \
                tuple(c.v_packed.shape) != (*c.k_norm.shape, self.d * c.v_bits // 8):
            raise ValueError("packed rows must be [n_pages, Hkv, page_size, d*bits/8]")
        self.views = (PagedCacheView * len(layers))(*(x.view() for x in layers))
        self.args = (self.Hkv, self.d, self.k_bits, self.v_bits)


@dataclass
class PageTable:
    """The books of a paged cache's pages (caller-owned device tensors, int32),
    and what the last call that wrote them said, unless it was given a tensor
    for that: a tensor of that call alone, on its stream."""
    block_table: torch.Tensor  # [n_seqs, max_pages]: page ids, -1 past a row's pages
    lens: torch.Tensor         # [n_seqs]: positions in use
    refs: torch.Tensor         # [n_pages]: holders of a page, 0 for a free one
    info: torch.Tensor | None = None      # [2]
    moved_to: torch.Tensor | None = None  # [n_pages], by tq_pages_compact

    @staticmethod
    def empty(n_seqs, max_pages, n_pages, device="cuda"):
        return PageTable(torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device),
                         torch.zeros(n_seqs, dtype=torch.int32, device=device),
                         torch.zeros(n_pages, dtype=torch.int32, device=device))

    def _view(self, layers: PagedLayers, shape) -> PageTableView:
        b, n, r = self.block_table, self.lens, self.refs
        _ints(layers.device, b, n, r)
        if b.shape != shape or n.numel() != shape[0] or r.numel() != layers.n_pages:
            raise ValueError("block_table [n_seqs, max_pages], lens [n_seqs], refs [n_pages] expected")
        return PageTableView(b.data_ptr(), n.data_ptr(), r.data_ptr())


_INT32 = torch.int32


def _ints(device, *ts):
    """Contiguous int32 CUDA tensors on `device`."""
    for t in ts:
        if t.dtype is not _INT32:
            raise TypeError("expected int32 tensors")
        if t.device != device or not t.is_contiguous():
            raise ValueError("expected contiguous CUDA tensors on one device")


def _raw_stream(device):
    """torch's current stream of the device, without a Stream object."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _same_device(device, *ts):
    for t in ts:
        if t.device != device:
            raise ValueError("all tensors must be on one device")


_STAY = nullcontext()


def _on(device):
    """The device made current for a call, where it is not."""
    return torch.cuda.device(device) if torch.cuda.current_device() != device.index else _STAY


def _layers(x) -> PagedLayers:
    return x if isinstance(x, PagedLayers) else PagedLayers(x)


def _scratch(workspace, device, bytes_fn, *sizes):
    """The workspace, or a new one of bytes_fn(*sizes) bytes."""
    if workspace is None:
        return torch.empty(max(bytes_fn(*sizes), 16), dtype=torch.uint8, device=device)
    if not workspace.is_cuda or not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be a contiguous CUDA tensor on the call's device")
    return workspace


def tq_pages_workspace_bytes(n_seqs: int, max_pages: int, n_pages: int) -> int:
    return int(lib().tq_pages_workspace_bytes(n_seqs, max_pages, n_pages))


_PAGES_COPY_FEW = 128  # TQ_PAGES_COPY_FEW: up to so many pairs need no workspace


def tq_pages_copy(src, dst, src_ids: torch.Tensor, dst_ids: torch.Tensor,
                  workspace: torch.Tensor | None = None):
    """Copy page src_ids[i] of `src` to page dst_ids[i] of `dst` (PagedLayers,
    a PagedCache or a list of them; one pool or two) in every layer.  Pairs
    with a negative id are skipped; a destination given twice, or that is also
    a source within one pool, is refused pair by pair (device status 62)."""
    src, dst = _layers(src), _layers(dst)
    if len(src.views) != len(dst.views) or src.args != dst.args or src.page_size != dst.page_size:
        raise ValueError("src and dst must have the same number of layers and geometry")
    _ints(dst.device, src_ids, dst_ids)
    if src_ids.numel() != dst_ids.numel():
        raise ValueError("src_ids and dst_ids must have one length")
    if src.device != dst.device:
        raise ValueError("src and dst must be on one device")
    n = src_ids.numel()
    with _on(dst.device):
        ws, size = None, 0
        if n > _PAGES_COPY_FEW or workspace is not None:
            ws = _scratch(workspace, dst.device, tq_pages_workspace_bytes, 0, 0, dst.n_pages)
            ws, size = ws.data_ptr(), ws.nbytes
        _check("tq_pages_copy", lib().tq_pages_copy(
            src.views, dst.views, len(dst.views), *dst.args, src_ids.data_ptr(), dst_ids.data_ptr(), n, ws, size,
            _raw_stream(dst.device)))


_FRESH: dict = {}  # per device, stream and length: int32 tensors that no call has had yet


def _fresh(device, stream, n):
    """A new int32 tensor [n], several to an allocation (one costs more than half
    of a small call); in a capture one of the graph's own memory."""
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(n, dtype=_INT32, device=device)
    key = (device.index, stream, n)
    try:
        return _FRESH[key].pop()
    except (KeyError, IndexError):  # none left, maybe since another thread took the last
        new = list(torch.empty(max(1, min(64, 65536 // n)), n, dtype=_INT32, device=device).unbind())
        first = new.pop()
        _FRESH[key] = new
        return first


def _pages(fn, table: PageTable, arg, layers, out, moved, info, workspace):
    layers = _layers(layers)
    shape = table.block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [n_seqs, max_pages]")
    n_seqs, max_pages = shape
    dev = layers.device
    with _on(dev):
        if out is None:
            out = PageTable(*(torch.empty_like(t) for t in (table.block_table, table.lens, table.refs)))
        a, b = table._view(layers, shape), out._view(layers, shape)
        stream = _raw_stream(dev)
        says, info = info is None, _fresh(dev, stream, 2) if info is None else info
        says_moved = arg is None and moved is None
        if says_moved:
            moved = _fresh(dev, stream, layers.n_pages)
        other = moved if arg is None else arg
        _ints(dev, info, other)
        if info.numel() != 2 or other.numel() != (layers.n_pages if arg is None else n_seqs):
            raise ValueError("info has 2 entries, parents and new_lens one per row, moved_to one per page")
        ws = _scratch(workspace, dev, tq_pages_workspace_bytes, n_seqs, max_pages, layers.n_pages)
        middle = (a, b, other.data_ptr()) if arg is None else (a, other.data_ptr(), b)
        _check(fn, getattr(lib(), fn)(*middle, n_seqs, max_pages, layers.views, len(layers.views), *layers.args,
                                      info.data_ptr(), ws.data_ptr(), ws.nbytes, stream))
        if says:
            out.info = info
        if says_moved:
            out.moved_to = moved
    return (out, info) if arg is not None else (out, moved, info)


def tq_pages_fork(table: PageTable, parents: torch.Tensor, layers, out: PageTable | None = None,
                  info: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Row i of the result is row parents[i] of `table` (int32; -1: empty):
    full pages shared, a partly filled last page copied for all children but
    one.  Returns (table, info [2]: pages taken, pages missing); without
    `info`, a new tensor, which the table keeps as its own."""
    return _pages("tq_pages_fork", table, parents, layers, out, None, info, workspace)


def tq_pages_resize(table: PageTable, new_lens: torch.Tensor, layers, out: PageTable | None = None,
                    info: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Row i gets the length new_lens[i] (int32; negative: unchanged): pages
    past it are given back, missing ones taken, and a shared last page that
    the row goes on in replaced by a private copy.  `out` may be `table`.
    Returns (table, info [2]: pages taken, pages missing), info as of
    tq_pages_fork."""
    return _pages("tq_pages_resize", table, new_lens, layers, out, None, info, workspace)


def tq_pages_compact(table: PageTable, layers, out: PageTable | None = None, moved_to: torch.Tensor | None = None,
                     info: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """The held pages moved to the lowest ids.  `out` may be `table`.  Returns
    (table, moved_to [n_pages]: each page's new id or -1, info [2]: pages
    held, pages moved); moved_to and info as of tq_pages_fork."""
    return _pages("tq_pages_compact", table, None, layers, out, moved_to, info, workspace)


def tq_device_status(reset: bool = False) -> int:
    st = ctypes.c_int(0)
    _check("tq_device_status", lib().tq_device_status(int(reset), ctypes.byref(st)))
    return st.value


# ------------------------------------------------------------ QJL residual keys

def tq_qjl_matrix(plan: Plan, device="cuda", out: torch.Tensor | None = None) -> torch.Tensor:
    """The plan's QJL projection S [d, d] fp32, drawn on the device."""
    if out is None:
        out = torch.empty(plan.d, plan.d, dtype=torch.float32, device=device)
    _cuda(out)
    _check("tq_qjl_matrix", lib().tq_qjl_matrix(plan.handle, out.data_ptr(), _stream(out)))
    return out


def tq_encode_qjl(plan: Plan, bits: int, S: torch.Tensor, x: torch.Tensor):
    """x: [n, d] fp32/bf16 -> (packed [n, d*bits/8] uint8, norms [n], rnorms [n] fp32)."""
    x2 = x.reshape(-1, plan.d)
    n = x2.shape[0]
    packed = torch.empty(n, plan.d * bits // 8, dtype=torch.uint8, device=x.device)
    norms = torch.empty(n, dtype=torch.float32, device=x.device)
    rnorms = torch.empty(n, dtype=torch.float32, device=x.device)
    _cuda(S, x2, packed, norms, rnorms)
    _check("tq_encode_qjl", lib().tq_encode_qjl(plan.handle, bits, S.data_ptr(), x2.data_ptr(), _dt(x2), n,
                                                packed.data_ptr(), norms.data_ptr(), rnorms.data_ptr(),
                                                _stream(x2)))
    return packed, norms, rnorms


def tq_decode_qjl(plan: Plan, bits: int, S: torch.Tensor, packed: torch.Tensor, norms: torch.Tensor,
                  rnorms: torch.Tensor, out_dtype=torch.float32) -> torch.Tensor:
    n = norms.numel()
    out = torch.empty(n, plan.d, dtype=out_dtype, device=packed.device)
    _cuda(S, packed, norms, rnorms, out)
    _check("tq_decode_qjl", lib().tq_decode_qjl(plan.handle, bits, S.data_ptr(), packed.data_ptr(),
                                                norms.data_ptr(), rnorms.data_ptr(), n, out.data_ptr(),
                                                _dt(out), _stream(out)))
    return out


def tq_attn_qjl_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, ctx_len: int) -> int:
    return int(lib().tq_attn_qjl_workspace_bytes(B, Hq, Hkv, d, ctx_len))


def tq_attn_decode_qjl(plan: Plan, S: torch.Tensor, q: torch.Tensor, cache: Cache, k_rnorm: torch.Tensor,
                       ctx_len: int, scale: float, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None) -> torch.Tensor:
    """q: [B, Hq, d] bf16; cache.k_* in the QJL format of cache.k_bits with
    k_rnorm [B, Hkv, cap] the gammas -> out [B, Hq, d] fp32."""
    B, Hq, d = q.shape
    Hkv = cache.k_norm.shape[1]
    if out is None:
        out = torch.empty(B, Hq, d, dtype=torch.float32, device=q.device)
    need = tq_attn_qjl_workspace_bytes(B, Hq, Hkv, d, ctx_len)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _cuda(S, q, k_rnorm, out, workspace)
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    _check("tq_attn_decode_qjl", lib().tq_attn_decode_qjl(
        plan.handle, S.data_ptr(), q.data_ptr(), B, Hq, Hkv, cache.view(), k_rnorm.data_ptr(), ctx_len,
        cache.k_bits, cache.v_bits, ctypes.c_float(scale), out.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream(q)))
    return out
