"""GB300 (sm_103a) decode attention: GQA query-head folding + Quest page sparsity.

A thin ctypes binding over the C ABI in ``include/gqaq.h`` (``libgqaq.so``).
Every function here only marshals arguments: it reads shapes and pointers
from torch tensors, builds a ``gqaq_dims``, passes
``torch.cuda.current_stream()`` and raises ``GqaqError`` on a non-zero status.
All arithmetic runs in the library's CUDA kernels. When the library is
missing, the import still succeeds but every call raises: there is no CPU
fallback.

Function names follow the C ABI: gqa_decode_attn, quest_append_kv,
quest_update_meta, quest_score_pages, quest_topk_pages, quest_sparse_attn,
quest_decode_attn, the 8-bit cache calls gqa_decode_attn_e4m3 /
kv_append_e4m3 and their Quest counterparts (quest_append_kv_e4m3,
quest_update_meta_e4m3, quest_score_pages_e4m3, quest_sparse_attn_e4m3), the
4-bit pair, prefill, and the paged serving calls (paged_build_tables,
paged_release_pages, paged_norm_rope_append, gqa_paged_attn, and the last two
over 8-bit pages: paged_norm_rope_append_e4m3, gqa_paged_attn_e4m3).
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqaq.so")

GQAQ_OK = 0
GQAQ_ERR_INVALID_ARG = 1
GQAQ_ERR_UNSUPPORTED = 2
GQAQ_ERR_WORKSPACE = 3
GQAQ_ERR_CUDA = 4
GQAQ_ERR_TIMEOUT = 5

GQAQ_DEV_TIMEOUT = 1
GQAQ_DEV_BAD_LEN = 2
GQAQ_DEV_BAD_PAGE = 4
GQAQ_DEV_BAD_POS = 8
GQAQ_DEV_NO_PAGES = 16

GQAQ_F16 = 0
GQAQ_BF16 = 1
GQAQ_PAGED_COUNTER_BYTES = 4096

GQAQ_OPT_MAX_CTAS = 1
GQAQ_OPT_WAIT_TIMEOUT_NS = 2
GQAQ_OPT_TEST_STALL = 3
GQAQ_OPT_CLUSTER_SIZE = 4
GQAQ_OPT_PDL = 5
GQAQ_OPT_QUEST_KERNEL = 6
GQAQ_OPT_PREFILL_SPLITS = 7
GQAQ_OPT_PREFILL_KERNEL = 8
GQAQ_OPT_QUEST_EARLY_META = 9
GQAQ_OPT_DENSE_EARLY_KV = 10

PAGE_SIZE = 16


class GqaqError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("max_len", ctypes.c_int), ("page_size", ctypes.c_int)]


class PagedDims(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int) for name in ("batch", "num_q_heads", "num_kv_heads", "head_dim", "page_size",
                                                  "num_pages", "max_pages", "max_tokens", "dtype", "max_len")]


# Exported symbols, in the order include/gqaq.h declares them.
EXPORTS = ("gqaq_workspace_bytes", "gqa_decode_attn", "quest_append_kv", "quest_update_meta",
           "quest_score_pages", "quest_topk_pages", "quest_sparse_attn", "quest_decode_attn",
           "gqa_decode_attn_noalloc", "gqa_decode_attn_e4m3", "kv_append_e4m3",
           "quest_append_kv_e4m3", "quest_update_meta_e4m3", "quest_score_pages_e4m3", "quest_sparse_attn_e4m3",
           "quest_decode_attn_e4m3",
           "gqa_decode_attn_int4", "kv_append_int4",
           "gqaq_prefill_workspace_bytes", "gqa_prefill_attn",
           "paged_build_tables", "paged_release_pages", "paged_norm_rope_append", "gqaq_paged_workspace_bytes",
           "gqa_paged_attn", "paged_norm_rope_append_e4m3", "gqa_paged_attn_e4m3",
           "gqaq_status_string", "gqaq_set_option", "gqaq_device_status", "gqaq_version")

_lib = None


def lib():
    """Load ``libgqaq.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, dp = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(Dims)
        L.gqaq_workspace_bytes.argtypes = [dp, i32]
        L.gqaq_workspace_bytes.restype = ctypes.c_size_t
        L.gqa_decode_attn.argtypes = [dp, vp, vp, vp, vp, ctypes.c_float, vp, vp, ctypes.c_size_t, vp]
        L.quest_append_kv.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp]
        L.quest_update_meta.argtypes = [dp, vp, vp, vp, i32, i32, vp]
        L.quest_score_pages.argtypes = [dp, vp, vp, vp, vp, vp]
        L.quest_topk_pages.argtypes = [dp, vp, vp, i32, vp, vp, ctypes.c_size_t, vp]
        L.quest_sparse_attn.argtypes = [dp, vp, vp, vp, vp, vp, i32, ctypes.c_float, vp, vp,
                                        ctypes.c_size_t, vp]
        L.quest_decode_attn.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, i32, ctypes.c_float, vp, vp, vp,
                                        vp, ctypes.c_size_t, vp]
        L.gqa_decode_attn_noalloc.argtypes = [dp, vp, vp, vp, vp, ctypes.c_float, vp, vp]
        f32 = ctypes.c_float
        L.gqa_decode_attn_e4m3.argtypes = [dp, vp, vp, vp, f32, f32, vp, f32, vp, vp, ctypes.c_size_t, vp]
        L.kv_append_e4m3.argtypes = [dp, vp, vp, vp, vp, vp, f32, f32, vp]
        L.quest_append_kv_e4m3.argtypes = [dp, vp, vp, vp, vp, vp, vp, f32, f32, vp]
        L.quest_update_meta_e4m3.argtypes = [dp, vp, vp, vp, i32, i32, vp]
        L.quest_score_pages_e4m3.argtypes = [dp, vp, vp, f32, vp, vp, vp]
        L.quest_sparse_attn_e4m3.argtypes = [dp, vp, vp, vp, f32, f32, vp, vp, i32, f32, vp, vp, ctypes.c_size_t, vp]
        L.quest_decode_attn_e4m3.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, f32, f32, f32, f32, vp, i32, f32, vp, vp,
                                             vp, vp]
        L.gqa_decode_attn_int4.argtypes = [dp, vp, vp, vp, vp, vp, vp, f32, vp, vp, ctypes.c_size_t, vp]
        L.kv_append_int4.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.gqaq_prefill_workspace_bytes.argtypes = [dp, i32]
        L.gqaq_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.gqa_prefill_attn.argtypes = [dp, i32, vp, vp, vp, vp, f32, vp, vp, ctypes.c_size_t, vp]
        pd, i64 = ctypes.POINTER(PagedDims), ctypes.c_int64
        L.paged_build_tables.argtypes = [pd] + [vp] * 11
        L.paged_release_pages.argtypes = [pd] + [vp] * 7
        L.paged_norm_rope_append.argtypes = [pd, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, f32, vp, i32, i32, i32, vp, vp,
                                             vp, vp]
        L.gqaq_paged_workspace_bytes.argtypes = [pd]
        L.gqaq_paged_workspace_bytes.restype = ctypes.c_size_t
        L.gqa_paged_attn.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, f32, vp, vp, ctypes.c_size_t, vp]
        L.paged_norm_rope_append_e4m3.argtypes = L.paged_norm_rope_append.argtypes[:-1] + [vp] * 3
        L.gqa_paged_attn_e4m3.argtypes = [pd, i32] + [vp] * 8 + [f32, vp, vp, ctypes.c_size_t, vp]
        L.gqaq_status_string.argtypes = [i32]
        L.gqaq_status_string.restype = ctypes.c_char_p
        L.gqaq_set_option.argtypes = [i32, ctypes.c_int64]
        L.gqaq_device_status.argtypes = [ctypes.POINTER(ctypes.c_int), i32]
        L.gqaq_version.argtypes = []
        for name in EXPORTS:
            if name not in ("gqaq_workspace_bytes", "gqaq_status_string", "gqaq_prefill_workspace_bytes",
                            "gqaq_paged_workspace_bytes"):
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gqaq_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != GQAQ_OK:
        raise GqaqError(fn, status, status_string(status))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(t: torch.Tensor, name: str, shape):
    """The library reads and writes whole buffers of these shapes: refuse any other."""
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _meta_shape(meta, B, Hkv, Lmax, D, page_size):
    _shape(meta, "meta", (B, Hkv, num_pages(Lmax, page_size), 2, D))


def _new_rows(k_new, v_new, pos, B, Hkv, D):
    _shape(k_new, "k_new", (B, Hkv, D))
    _shape(v_new, "v_new", (B, Hkv, D))
    _shape(pos, "pos", (B,))


def make_dims(batch, num_q_heads, num_kv_heads, head_dim, max_len, page_size=PAGE_SIZE) -> Dims:
    return Dims(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(max_len),
                int(page_size))


def dims_of(q: torch.Tensor, k_cache: torch.Tensor, page_size: int = PAGE_SIZE) -> Dims:
    B, Hq, D = q.shape
    _, Hkv, Lmax, _ = k_cache.shape
    return make_dims(B, Hq, Hkv, D, Lmax, page_size)


def set_option(option: int, value: int):
    _check("gqaq_set_option", lib().gqaq_set_option(int(option), int(value)))


def device_status(reset: bool = True) -> int:
    """Return the current device's GQAQ_DEV_* flags (synchronises the device)."""
    flags = ctypes.c_int(0)
    rc = lib().gqaq_device_status(ctypes.byref(flags), 1 if reset else 0)
    if rc not in (GQAQ_OK, GQAQ_ERR_TIMEOUT):
        _check("gqaq_device_status", rc)
    return flags.value


def workspace_bytes(dims: Dims, max_selected_pages: int = 0) -> int:
    n = lib().gqaq_workspace_bytes(ctypes.byref(dims), int(max_selected_pages))
    if n == 0:
        raise GqaqError("gqaq_workspace_bytes", GQAQ_ERR_UNSUPPORTED, "dims rejected")
    return int(n)


def alloc_workspace(dims: Dims, device, max_selected_pages: int = 0) -> torch.Tensor:
    """Workspace for gqa_decode_attn / quest_sparse_attn, and with
    max_selected_pages = k also for quest_decode_attn's work-queue kernel.
    Zero-filled once, as the library asks; every call leaves its counters at
    zero again."""
    return torch.zeros(workspace_bytes(dims, max_selected_pages), dtype=torch.uint8, device=device)


def workspace_zero_bytes(dims: Dims) -> int:
    """Leading bytes of a workspace that hold counters and flags (zero between calls)."""
    return (256 + 12 * dims.batch * dims.num_kv_heads + 255) // 256 * 256


def num_pages(max_len: int, page_size: int = PAGE_SIZE) -> int:
    return (int(max_len) + page_size - 1) // page_size


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------
def gqa_decode_attn(q, k_cache, v_cache, valid_len, scale: float, out=None, workspace=None):
    """Dense folded-GQA decode attention. q [B,Hq,D], caches [B,Hkv,Lmax,D] fp16."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(v_cache, "v_cache", torch.float16, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    d = dims_of(q, k_cache)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if workspace is None:
        workspace = alloc_workspace(d, q.device)
    _check("gqa_decode_attn", lib().gqa_decode_attn(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(valid_len), float(scale),
        _ptr(out), _ptr(workspace), workspace.numel(), _stream(q)))
    return out


def quest_decode_attn(q, k_cache, v_cache, meta, valid_len, k: int, scale: float, k_new=None, v_new=None,
                      pos=None, out=None, scores=None, page_idx=None, page_size: int = PAGE_SIZE,
                      workspace=None):
    """Fused Quest step in one launch: optional append (k_new, v_new at pos),
    page scores, top-k pages and attention over them. scores/page_idx are
    optional outputs. With a workspace (alloc_workspace(dims, device, k)) the
    step runs as one GPU-wide work queue; without, one cluster per unit."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(v_cache, "v_cache", torch.float16, 4)
    _need(meta, "meta", torch.float16, 5)
    _need(valid_len, "valid_len", torch.int32, 1)
    if pos is not None:
        _need(k_new, "k_new", torch.float16, 3)
        _need(v_new, "v_new", torch.float16, 3)
        _need(pos, "pos", torch.int32, 1)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if scores is not None:
        _need(scores, "scores", torch.float32, 3)
    if page_idx is not None:
        _need(page_idx, "page_idx", torch.int32, 3)
    d = dims_of(q, k_cache, page_size)
    _meta_shape(meta, d.batch, d.num_kv_heads, d.max_len, d.head_dim, page_size)
    _shape(valid_len, "valid_len", (d.batch,))
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    if pos is not None:
        _new_rows(k_new, v_new, pos, d.batch, d.num_kv_heads, d.head_dim)
    if scores is not None:
        _shape(scores, "scores", (d.batch, d.num_kv_heads, num_pages(d.max_len, page_size)))
    if page_idx is not None:
        _shape(page_idx, "page_idx", (d.batch, d.num_kv_heads, int(k)))
    _check("quest_decode_attn", lib().quest_decode_attn(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(meta), _ptr(k_new), _ptr(v_new),
        _ptr(pos), _ptr(valid_len), int(k), float(scale), _ptr(out), _ptr(scores), _ptr(page_idx),
        _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(q)))
    return out


def gqa_decode_attn_noalloc(q, k_cache, v_cache, valid_len, scale: float, out):
    """gqa_decode_attn without a workspace, for callers that cannot allocate
    device memory (the library keeps the scratch in its own fixed 1 MiB array).
    ``out`` must be given. Overlapping calls race on the shared scratch."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(v_cache, "v_cache", torch.float16, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    _need(out, "out", torch.float16, 3)
    d = dims_of(q, k_cache)
    _check("gqa_decode_attn_noalloc", lib().gqa_decode_attn_noalloc(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(valid_len), float(scale),
        _ptr(out), _stream(q)))
    return out


def gqa_decode_attn_e4m3(q, k_cache, v_cache, k_scale: float, v_scale: float, valid_len, scale: float,
                         out=None, workspace=None):
    """Dense folded-GQA decode attention over an E4M3 cache: k_cache / v_cache
    [B,Hkv,Lmax,D] uint8 codes, dequantized as code value * k_scale (v_scale)."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    d = dims_of(q, k_cache)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if workspace is None:
        workspace = alloc_workspace(d, q.device)
    _check("gqa_decode_attn_e4m3", lib().gqa_decode_attn_e4m3(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), _ptr(valid_len),
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _stream(q)))
    return out


def kv_append_e4m3(k_cache, v_cache, k_new, v_new, pos, k_inv_scale: float, v_inv_scale: float):
    """Quantize k_new/v_new [B,Hkv,D] fp16 to E4M3 (x * inv_scale, nearest-even,
    saturating) and write the codes at row pos[b] of the uint8 caches."""
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(k_new, "k_new", torch.float16, 3)
    _need(v_new, "v_new", torch.float16, 3)
    _need(pos, "pos", torch.int32, 1)
    B, Hkv, Lmax, D = k_cache.shape
    d = make_dims(B, Hkv, Hkv, D, Lmax)
    _check("kv_append_e4m3", lib().kv_append_e4m3(
        ctypes.byref(d), _ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(pos), float(k_inv_scale),
        float(v_inv_scale), _stream(k_cache)))


def new_meta_e4m3(batch: int, num_kv_heads: int, max_len: int, head_dim: int, device,
                  page_size: int = PAGE_SIZE) -> torch.Tensor:
    """Allocate E4M3 page bounds [B,Hkv,Pmax,2,D] uint8 (contents undefined)."""
    return torch.empty(batch, num_kv_heads, num_pages(max_len, page_size), 2, head_dim, dtype=torch.uint8,
                       device=device)


def quest_append_kv_e4m3(k_cache, v_cache, meta, k_new, v_new, pos, k_inv_scale: float, v_inv_scale: float,
                         page_size: int = PAGE_SIZE):
    """kv_append_e4m3 plus the page's E4M3 bounds (meta [B,Hkv,Pmax,2,D] uint8)."""
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(meta, "meta", torch.uint8, 5)
    _need(k_new, "k_new", torch.float16, 3)
    _need(v_new, "v_new", torch.float16, 3)
    _need(pos, "pos", torch.int32, 1)
    B, Hkv, Lmax, D = k_cache.shape
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    _meta_shape(meta, B, Hkv, Lmax, D, page_size)
    _new_rows(k_new, v_new, pos, B, Hkv, D)
    d = make_dims(B, Hkv, Hkv, D, Lmax, page_size)
    _check("quest_append_kv_e4m3", lib().quest_append_kv_e4m3(
        ctypes.byref(d), _ptr(k_cache), _ptr(v_cache), _ptr(meta), _ptr(k_new), _ptr(v_new), _ptr(pos),
        float(k_inv_scale), float(v_inv_scale), _stream(k_cache)))


def quest_update_meta_e4m3(k_cache, valid_len, meta, page_begin: int = 0, page_end: Optional[int] = None,
                           page_size: int = PAGE_SIZE):
    """Rebuild the E4M3 page bounds of pages [page_begin, page_end) from the cache codes."""
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    _need(meta, "meta", torch.uint8, 5)
    B, Hkv, Lmax, D = k_cache.shape
    _meta_shape(meta, B, Hkv, Lmax, D, page_size)
    _shape(valid_len, "valid_len", (B,))
    d = make_dims(B, Hkv, Hkv, D, Lmax, page_size)
    if page_end is None:
        page_end = num_pages(Lmax, page_size)
    _check("quest_update_meta_e4m3", lib().quest_update_meta_e4m3(
        ctypes.byref(d), _ptr(k_cache), _ptr(valid_len), _ptr(meta), int(page_begin), int(page_end),
        _stream(k_cache)))
    return meta


def quest_score_pages_e4m3(q, meta, k_scale: float, valid_len, max_len: int, scores=None,
                           page_size: int = PAGE_SIZE):
    """k_scale * U(p,q) from E4M3 page bounds -> scores [B,Hkv,Pmax] fp32."""
    _need(q, "q", torch.float16, 3)
    _need(meta, "meta", torch.uint8, 5)
    _need(valid_len, "valid_len", torch.int32, 1)
    B, Hq, D = q.shape
    Hkv = meta.shape[1]
    d = make_dims(B, Hq, Hkv, D, max_len, page_size)
    _meta_shape(meta, B, Hkv, max_len, D, page_size)
    _shape(valid_len, "valid_len", (B,))
    if scores is None:
        scores = torch.empty(B, Hkv, num_pages(max_len, page_size), dtype=torch.float32, device=q.device)
    _need(scores, "scores", torch.float32, 3)
    _shape(scores, "scores", (B, Hkv, num_pages(max_len, page_size)))
    _check("quest_score_pages_e4m3", lib().quest_score_pages_e4m3(
        ctypes.byref(d), _ptr(q), _ptr(meta), float(k_scale), _ptr(valid_len), _ptr(scores), _stream(q)))
    return scores


def quest_sparse_attn_e4m3(q, k_cache, v_cache, k_scale: float, v_scale: float, valid_len, page_idx, scale: float,
                           out=None, workspace=None, page_size: int = PAGE_SIZE):
    """Attention over the selected pages of an E4M3 cache (page_idx [B,Hkv,k])."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    _need(page_idx, "page_idx", torch.int32, 3)
    d = dims_of(q, k_cache, page_size)
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    _shape(valid_len, "valid_len", (d.batch,))
    _shape(page_idx, "page_idx", (d.batch, d.num_kv_heads, page_idx.shape[2]))
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if workspace is None:
        workspace = alloc_workspace(d, q.device)
    _check("quest_sparse_attn_e4m3", lib().quest_sparse_attn_e4m3(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), _ptr(valid_len),
        _ptr(page_idx), int(page_idx.shape[2]), float(scale), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(q)))
    return out


def quest_decode_attn_e4m3(q, k_cache, v_cache, meta, valid_len, k: int, scale: float, k_scale: float,
                           v_scale: float, k_new=None, v_new=None, pos=None, k_inv_scale: float = 1.0,
                           v_inv_scale: float = 1.0, out=None, scores=None, page_idx=None,
                           page_size: int = PAGE_SIZE):
    """quest_decode_attn over an E4M3 cache (codes [B,Hkv,Lmax,D] uint8, bounds
    [B,Hkv,Pmax,2,D] uint8) in one launch; the optional append quantizes
    k_new/v_new with k_inv_scale / v_inv_scale."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.uint8, 4)
    _need(v_cache, "v_cache", torch.uint8, 4)
    _need(meta, "meta", torch.uint8, 5)
    _need(valid_len, "valid_len", torch.int32, 1)
    d = dims_of(q, k_cache, page_size)
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    _meta_shape(meta, d.batch, d.num_kv_heads, d.max_len, d.head_dim, page_size)
    _shape(valid_len, "valid_len", (d.batch,))
    if pos is not None:
        _need(k_new, "k_new", torch.float16, 3)
        _need(v_new, "v_new", torch.float16, 3)
        _need(pos, "pos", torch.int32, 1)
        _new_rows(k_new, v_new, pos, d.batch, d.num_kv_heads, d.head_dim)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if scores is not None:
        _need(scores, "scores", torch.float32, 3)
        _shape(scores, "scores", (d.batch, d.num_kv_heads, num_pages(d.max_len, page_size)))
    if page_idx is not None:
        _need(page_idx, "page_idx", torch.int32, 3)
        _shape(page_idx, "page_idx", (d.batch, d.num_kv_heads, int(k)))
    _check("quest_decode_attn_e4m3", lib().quest_decode_attn_e4m3(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(meta), _ptr(k_new), _ptr(v_new), _ptr(pos),
        float(k_inv_scale), float(v_inv_scale), float(k_scale), float(v_scale), _ptr(valid_len), int(k),
        float(scale), _ptr(out), _ptr(scores), _ptr(page_idx), _stream(q)))
    return out


def prefill_workspace_bytes(dims: Dims, q_len: int) -> int:
    n = lib().gqaq_prefill_workspace_bytes(ctypes.byref(dims), int(q_len))
    if n == 0:
        raise GqaqError("gqaq_prefill_workspace_bytes", GQAQ_ERR_UNSUPPORTED, "dims rejected")
    return int(n)


def alloc_prefill_workspace(dims: Dims, q_len: int, device) -> torch.Tensor:
    """Zero-filled workspace for gqa_prefill_attn (its counters stay zero between calls)."""
    return torch.zeros(prefill_workspace_bytes(dims, q_len), dtype=torch.uint8, device=device)


def gqa_prefill_attn(q, k_cache, v_cache, start, scale: float, out=None, workspace=None):
    """Causal attention of a chunk: q [B,Hq,q_len,D], caches [B,Hkv,Lmax,D]
    holding the chunk at rows start[b] .. start[b]+q_len-1; token t attends to
    rows 0 .. start[b]+t. The G heads and q_len tokens of a KV head are one
    folded row block."""
    _need(q, "q", torch.float16, 4)
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(v_cache, "v_cache", torch.float16, 4)
    _need(start, "start", torch.int32, 1)
    B, Hq, q_len, D = q.shape
    _, Hkv, Lmax, _ = k_cache.shape
    d = make_dims(B, Hq, Hkv, D, Lmax)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 4)
    if workspace is None:
        workspace = alloc_prefill_workspace(d, q_len, q.device)
    _check("gqa_prefill_attn", lib().gqa_prefill_attn(
        ctypes.byref(d), int(q_len), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(start), float(scale), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(q)))
    return out


def gqa_decode_attn_int4(q, k_codes, k_scales, v_codes, v_scales, valid_len, scale: float, out=None,
                         workspace=None):
    """Dense folded-GQA decode attention over a 4-bit cache: codes
    [B,Hkv,Lmax,D/2] uint8 (two levels + 8 per byte, low nibble first), scales
    [B,Hkv,Lmax] fp32 (value = level * scale). Lmax must be a multiple of 4."""
    _need(q, "q", torch.float16, 3)
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        _need(t, name, torch.uint8, 4)
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _need(t, name, torch.float32, 3)
    _need(valid_len, "valid_len", torch.int32, 1)
    B, Hq, D = q.shape
    _, Hkv, Lmax, _ = k_codes.shape
    d = make_dims(B, Hq, Hkv, D, Lmax)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if workspace is None:
        workspace = alloc_workspace(d, q.device)
    _check("gqa_decode_attn_int4", lib().gqa_decode_attn_int4(
        ctypes.byref(d), _ptr(q), _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _ptr(valid_len),
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _stream(q)))
    return out


def kv_append_int4(k_codes, k_scales, v_codes, v_scales, k_new, v_new, pos):
    """Quantize k_new/v_new [B,Hkv,D] fp16 rows to INT4 (scale = amax / 7 per
    row) and write codes and scales at row pos[b]."""
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        _need(t, name, torch.uint8, 4)
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _need(t, name, torch.float32, 3)
    _need(k_new, "k_new", torch.float16, 3)
    _need(v_new, "v_new", torch.float16, 3)
    _need(pos, "pos", torch.int32, 1)
    B, Hkv, Lmax, _ = k_codes.shape
    D = k_new.shape[2]
    d = make_dims(B, Hkv, Hkv, D, Lmax)
    _check("kv_append_int4", lib().kv_append_int4(
        ctypes.byref(d), _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _ptr(k_new), _ptr(v_new),
        _ptr(pos), _stream(k_codes)))


def quest_append_kv(k_cache, v_cache, meta, k_new, v_new, pos, page_size: int = PAGE_SIZE):
    """Write k_new/v_new [B,Hkv,D] at row pos[b] and update that page's min/max."""
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(v_cache, "v_cache", torch.float16, 4)
    _need(meta, "meta", torch.float16, 5)
    _need(k_new, "k_new", torch.float16, 3)
    _need(v_new, "v_new", torch.float16, 3)
    _need(pos, "pos", torch.int32, 1)
    B, Hkv, Lmax, D = k_cache.shape
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    _meta_shape(meta, B, Hkv, Lmax, D, page_size)
    _new_rows(k_new, v_new, pos, B, Hkv, D)
    d = make_dims(B, Hkv, Hkv, D, Lmax, page_size)
    _check("quest_append_kv", lib().quest_append_kv(
        ctypes.byref(d), _ptr(k_cache), _ptr(v_cache), _ptr(meta), _ptr(k_new), _ptr(v_new),
        _ptr(pos), _stream(k_cache)))


def quest_update_meta(k_cache, valid_len, meta, page_begin: int = 0, page_end: Optional[int] = None,
                      page_size: int = PAGE_SIZE):
    """Rebuild page min/max [B,Hkv,Pmax,2,D] for pages [page_begin, page_end)."""
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    _need(meta, "meta", torch.float16, 5)
    B, Hkv, Lmax, D = k_cache.shape
    _meta_shape(meta, B, Hkv, Lmax, D, page_size)
    _shape(valid_len, "valid_len", (B,))
    d = make_dims(B, Hkv, Hkv, D, Lmax, page_size)
    if page_end is None:
        page_end = num_pages(Lmax, page_size)
    _check("quest_update_meta", lib().quest_update_meta(
        ctypes.byref(d), _ptr(k_cache), _ptr(valid_len), _ptr(meta), int(page_begin), int(page_end),
        _stream(k_cache)))
    return meta


def quest_score_pages(q, meta, valid_len, max_len: int, scores=None, page_size: int = PAGE_SIZE):
    """U(p,q) per KV head (max over its G folded query rows) -> scores [B,Hkv,Pmax] fp32."""
    _need(q, "q", torch.float16, 3)
    _need(meta, "meta", torch.float16, 5)
    _need(valid_len, "valid_len", torch.int32, 1)
    B, Hq, D = q.shape
    Hkv = meta.shape[1]
    d = make_dims(B, Hq, Hkv, D, max_len, page_size)
    _meta_shape(meta, B, Hkv, max_len, D, page_size)
    _shape(valid_len, "valid_len", (B,))
    if scores is None:
        scores = torch.empty(B, Hkv, num_pages(max_len, page_size), dtype=torch.float32, device=q.device)
    _need(scores, "scores", torch.float32, 3)
    _shape(scores, "scores", (B, Hkv, num_pages(max_len, page_size)))
    _check("quest_score_pages", lib().quest_score_pages(
        ctypes.byref(d), _ptr(q), _ptr(meta), _ptr(valid_len), _ptr(scores), _stream(q)))
    return scores


def quest_topk_pages(scores, valid_len, k: int, max_len: int, page_idx=None, page_size: int = PAGE_SIZE):
    """Top-k pages per (b, kv) -> page_idx [B,Hkv,k] int32, ascending, -1 padded."""
    _need(scores, "scores", torch.float32, 3)
    _need(valid_len, "valid_len", torch.int32, 1)
    B, Hkv, _ = scores.shape
    _shape(scores, "scores", (B, Hkv, num_pages(max_len, page_size)))
    _shape(valid_len, "valid_len", (B,))
    d = make_dims(B, Hkv, Hkv, 64, max_len, page_size)
    if page_idx is None:
        page_idx = torch.empty(B, Hkv, int(k), dtype=torch.int32, device=scores.device)
    _need(page_idx, "page_idx", torch.int32, 3)
    _shape(page_idx, "page_idx", (B, Hkv, int(k)))
    _check("quest_topk_pages", lib().quest_topk_pages(
        ctypes.byref(d), _ptr(scores), _ptr(valid_len), int(k), _ptr(page_idx), None, 0,
        _stream(scores)))
    return page_idx


def quest_sparse_attn(q, k_cache, v_cache, valid_len, page_idx, scale: float, out=None, workspace=None,
                      page_size: int = PAGE_SIZE):
    """Attention over the selected pages only (page_idx [B,Hkv,k])."""
    _need(q, "q", torch.float16, 3)
    _need(k_cache, "k_cache", torch.float16, 4)
    _need(v_cache, "v_cache", torch.float16, 4)
    _need(valid_len, "valid_len", torch.int32, 1)
    _need(page_idx, "page_idx", torch.int32, 3)
    d = dims_of(q, k_cache, page_size)
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    _shape(valid_len, "valid_len", (d.batch,))
    _shape(page_idx, "page_idx", (d.batch, d.num_kv_heads, page_idx.shape[2]))
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float16, 3)
    if workspace is None:
        workspace = alloc_workspace(d, q.device)
    _check("quest_sparse_attn", lib().quest_sparse_attn(
        ctypes.byref(d), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(valid_len), _ptr(page_idx),
        int(page_idx.shape[2]), float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _stream(q)))
    return out


def new_meta(batch: int, num_kv_heads: int, max_len: int, head_dim: int, device,
             page_size: int = PAGE_SIZE) -> torch.Tensor:
    """Allocate a metadata buffer [B,Hkv,Pmax,2,D] fp16 (contents undefined)."""
    return torch.empty(batch, num_kv_heads, num_pages(max_len, page_size), 2, head_dim,
                       dtype=torch.float16, device=device)


# ---------------------------------------------------------------------------
# Paged caches
# ---------------------------------------------------------------------------
_PAGED_DTYPES = {torch.float16: GQAQ_F16, torch.bfloat16: GQAQ_BF16}


def _int32(name: str, value) -> int:
    """value, where the library's 32-bit argument can hold it (ctypes would cut it short)."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def make_paged_dims(batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages, max_tokens,
                    dtype=torch.float16, max_len: int = 0) -> PagedDims:
    """Shape of a paged step; dtype is torch.float16 or torch.bfloat16. max_len limits a request's tokens in the
    plan (0: what max_pages hold)."""
    if dtype not in _PAGED_DTYPES:
        raise ValueError(f"paged caches hold torch.float16 or torch.bfloat16, not {dtype}")
    return PagedDims(*(_int32(name, int(value)) for (name, _), value in zip(
        PagedDims._fields_, (batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages, max_tokens,
                             _PAGED_DTYPES[dtype], max_len))))


def paged_dims_of(q: torch.Tensor, k_pages: torch.Tensor, block_table: torch.Tensor) -> PagedDims:
    T, Hq, D = q.shape
    num_pages, Hkv, S, _ = k_pages.shape
    B, max_pages = block_table.shape
    return make_paged_dims(B, Hq, Hkv, D, S, num_pages, max_pages, T, q.dtype)


def paged_workspace_bytes(dims: PagedDims) -> int:
    n = lib().gqaq_paged_workspace_bytes(ctypes.byref(dims))
    if n == 0:
        raise GqaqError("gqaq_paged_workspace_bytes", GQAQ_ERR_UNSUPPORTED, "dims rejected")
    return int(n)


def alloc_paged_workspace(dims: PagedDims, device) -> torch.Tensor:
    """Zero-filled workspace for gqa_paged_attn (its counters stay zero between calls).
    Its size depends on head_dim and the device only, so one serves every batch and every layer in a stream."""
    return torch.zeros(paged_workspace_bytes(dims), dtype=torch.uint8, device=device)


def _paged_workspace_of_one_call(dims: PagedDims, device) -> torch.Tensor:
    """A workspace with zeros where the library needs them: filling all 40 MB would take longer than many calls."""
    workspace = torch.empty(paged_workspace_bytes(dims), dtype=torch.uint8, device=device)
    workspace[:GQAQ_PAGED_COUNTER_BYTES].zero_()
    return workspace


def new_pages(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device,
              dtype=torch.float16) -> torch.Tensor:
    """Allocate one pool of pages [num_pages,Hkv,S,D] (contents undefined)."""
    return torch.empty(num_pages, num_kv_heads, page_size, head_dim, dtype=dtype, device=device)


def new_pages_e4m3(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device):
    """Allocate one pool of 8-bit pages: E4M3 codes [num_pages,Hkv,S,D] uint8 (contents undefined) and the pages'
    exponents [num_pages,Hkv] int8 (zeros); a channel's value is value(code) * 2^exponent."""
    return (torch.empty(num_pages, num_kv_heads, page_size, head_dim, dtype=torch.uint8, device=device),
            torch.zeros(num_pages, num_kv_heads, dtype=torch.int8, device=device))


def _paged_bad(name: str, t, dtype, shape, dev: int):
    """Say what _paged found wrong with an argument."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device cuda:{dev}, got {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _paged(name: str, t, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this dtype and shape on the current device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _paged_bad(name, t, dtype, shape, dev)


def _paged_dim(name: str, t, ndim: int):
    """The shape of a tensor argument of ndim dims."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t.shape


def _paged_device(name: str, t) -> int:
    """The current device, which must hold t (and with it every other argument)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if dev != _cuda_device():
        raise ValueError(f"{name} must be on the current device, got {t.device}")
    return dev


@functools.lru_cache(maxsize=1024)
def _paged_dims_ref(*fields):
    """A pointer to the gqaq_paged_dims with these fields (the library only reads it during the call)."""
    return ctypes.pointer(PagedDims(*(_int32(name, value) for (name, _), value in zip(PagedDims._fields_, fields))))


_cuda_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_cuda_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def paged_build_tables(cache_len, new_len, free_pages, free_count, block_table, max_tokens: int,
                       page_size: int = PAGE_SIZE, kv_len=None, cu_q=None, positions=None, slots=None,
                       free_count_out=None, max_len: int = 0):
    """Plan a paged step on the GPU from cache_len / new_len [B]: take pages off the end of
    free_pages[:free_count], write them to block_table [B,max_pages], and return
    (kv_len [B], cu_q [B+1], positions [max_tokens], slots [max_tokens], free_count_out [1]), all int32.
    Requests are served in order, each wholly or not at all; a refused one has kv_len 0 and slots -1.
    max_len is the most tokens of a request (0: what its row of block_table holds).
    free_count_out may be free_count itself; without it a new tensor holds the count."""
    i32 = torch.int32
    (B,) = _paged_dim("cache_len", cache_len, 1)
    dev = _paged_device("cache_len", cache_len)
    _, width = _paged_dim("block_table", block_table, 2)
    (pool,) = _paged_dim("free_pages", free_pages, 1)
    T, per_b, per_t, one = int(max_tokens), (B,), (int(max_tokens),), (1,)
    if kv_len is None:
        kv_len = torch.empty(per_b, dtype=i32, device=cache_len.device)
    if cu_q is None:
        cu_q = torch.empty(B + 1, dtype=i32, device=cache_len.device)
    if positions is None:
        positions = torch.empty(per_t, dtype=i32, device=cache_len.device)
    if slots is None:
        slots = torch.empty(per_t, dtype=i32, device=cache_len.device)
    if free_count_out is None:
        free_count_out = torch.empty(one, dtype=i32, device=cache_len.device)
    status = lib().paged_build_tables(
        _paged_dims_ref(B, 0, 0, 0, int(page_size), pool, width, T, 0, int(max_len)),
        _paged("cache_len", cache_len, i32, per_b, dev), _paged("new_len", new_len, i32, per_b, dev),
        _paged("free_pages", free_pages, i32, (pool,), dev), _paged("free_count", free_count, i32, one, dev),
        _paged("block_table", block_table, i32, (B, width), dev), _paged("kv_len", kv_len, i32, per_b, dev),
        _paged("cu_q", cu_q, i32, (B + 1,), dev), _paged("positions", positions, i32, per_t, dev),
        _paged("slots", slots, i32, per_t, dev), _paged("free_count_out", free_count_out, i32, one, dev),
        _cuda_stream(dev))
    if status:
        _check("paged_build_tables", status)
    return kv_len, cu_q, positions, slots, free_count_out


def paged_release_pages(kv_len, keep_len, block_table, free_pages, free_count, page_size: int = PAGE_SIZE,
                        free_count_out=None):
    """Append the pages past keep_len [B] of kv_len [B] tokens to free_pages behind its first free_count
    entries; returns the new count (free_count_out, which may be free_count itself)."""
    i32 = torch.int32
    (B,) = _paged_dim("kv_len", kv_len, 1)
    dev = _paged_device("kv_len", kv_len)
    _, width = _paged_dim("block_table", block_table, 2)
    (pool,) = _paged_dim("free_pages", free_pages, 1)
    if free_count_out is None:
        free_count_out = torch.empty(1, dtype=i32, device=kv_len.device)
    status = lib().paged_release_pages(
        _paged_dims_ref(B, 0, 0, 0, int(page_size), pool, width, 1, 0),
        _paged("kv_len", kv_len, i32, (B,), dev), _paged("keep_len", keep_len, i32, (B,), dev),
        _paged("block_table", block_table, i32, (B, width), dev), _paged("free_pages", free_pages, i32, (pool,), dev),
        _paged("free_count", free_count, i32, (1,), dev), _paged("free_count_out", free_count_out, i32, (1,), dev),
        _cuda_stream(dev))
    if status:
        _check("paged_release_pages", status)
    return free_count_out


def _paged_rows(name: str, t, dtype, shape, dev: int):
    """(address, elements between tokens) of [T,H,D] rows whose heads are contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _paged_bad(name, t, dtype, shape, dev)
    st, sh, sd = t.stride()
    if sd != 1 or (sh != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {(st, sh, sd)}")
    return t.data_ptr(), st if shape[0] > 1 else shape[1] * shape[2]  # a single token: whatever the stride says


def _paged_append(fn, q, k, v, positions, slots, pools, pool_dtype, exps, q_weight, k_weight, eps, cos_sin, interleaved, q_out):
    """The append named fn; pools: k_pages and v_pages, exps: k_exp and v_exp of 8-bit pages."""
    i32 = torch.int32
    q_rows = T, Hq, D = _paged_dim("q", q, 3)
    dev = _paged_device("q", q)
    pool = num_pages, Hkv, S, _ = _paged_dim("k_pages", pools[0], 4)
    per_t, kv_rows, dt = (T,), (T, Hkv, D), q.dtype
    if dt not in _PAGED_DTYPES:
        raise ValueError(f"q must be torch.float16 or torch.bfloat16, got {dt}")
    if q_out is None:
        q_out = torch.empty(q_rows, dtype=dt, device=q.device)
    aq, sq = _paged_rows("q", q, dt, q_rows, dev)
    ak, sk = _paged_rows("k", k, dt, kv_rows, dev)
    av, sv = _paged_rows("v", v, dt, kv_rows, dev)
    cs, rope, most = None, 0, 0
    if cos_sin is not None:
        most, rope = angles = _paged_dim("cos_sin", cos_sin, 2)
        cs = _paged("cos_sin", cos_sin, torch.float32, angles, dev)
    pool_dtype = pool_dtype or dt
    more = ()
    if exps:
        per_page = (num_pages, Hkv)
        more = _paged("k_exp", exps[0], torch.int8, per_page, dev), _paged("v_exp", exps[1], torch.int8, per_page, dev)
    status = getattr(lib(), fn)(
        _paged_dims_ref(1, Hq, Hkv, D, S, num_pages, 1, T, _PAGED_DTYPES[dt]), aq, sq, ak, sk, av, sv,
        _paged("positions", positions, i32, per_t, dev), _paged("slots", slots, i32, per_t, dev),
        None if q_weight is None else _paged("q_weight", q_weight, dt, (D,), dev),
        None if k_weight is None else _paged("k_weight", k_weight, dt, (D,), dev), eps, cs, rope, most,
        1 if interleaved else 0, _paged("q_out", q_out, dt, q_rows, dev),
        _paged("k_pages", pools[0], pool_dtype, (num_pages, Hkv, S, D), dev), _paged("v_pages", pools[1], pool_dtype, pool, dev),
        *more, _cuda_stream(dev))
    if status:
        _check(fn, status)
    return q_out


def paged_norm_rope_append(q, k, v, positions, slots, k_pages, v_pages, q_weight=None, k_weight=None,
                           eps: float = 1e-6, cos_sin=None, interleaved: bool = False, q_out=None):
    """Per-head RMS norms of q [T,Hq,D] and k [T,Hkv,D] (weights [D], each optional), rotary positions by
    cos_sin [max_position,rope_dim] fp32 (cosines, then sines; None: no rotation), and the append: q to
    q_out [T,Hq,D], k and v to row slots[t] of the pages [num_pages,Hkv,S,D]. Tokens with slots[t] < 0
    are padding. q, k and v may be slices of one fused projection (heads contiguous, any token stride
    that is a multiple of 8). Returns q_out."""
    return _paged_append("paged_norm_rope_append", q, k, v, positions, slots, (k_pages, v_pages), None, (), q_weight, k_weight, eps,
                         cos_sin, interleaved, q_out)


def paged_norm_rope_append_e4m3(q, k, v, positions, slots, k_pages, v_pages, k_exp, v_exp, q_weight=None, k_weight=None,
                                eps: float = 1e-6, cos_sin=None, interleaved: bool = False, q_out=None):
    """paged_norm_rope_append to 8-bit pages (codes uint8, exponents [num_pages,Hkv] int8; see new_pages_e4m3): a
    page's exponent covers its largest magnitude. Rows that join a page may raise it, and the codes there are then
    rounded again; rows from a page's first one on start it afresh, and until then it never falls, also when the rows
    that raised it have been released. Infinities become the page's largest number; NaN stays. The tokens of a page lie
    one behind the other."""
    return _paged_append("paged_norm_rope_append_e4m3", q, k, v, positions, slots, (k_pages, v_pages), torch.uint8, (k_exp, v_exp),
                         q_weight, k_weight, eps, cos_sin, interleaved, q_out)


def _paged_attn(fn, q, pools, pool_dtype, exps, block_table, cu_q, kv_len, scale, max_q_len, out, workspace):
    """The attention named fn; pools: k_pages and v_pages, exps: k_exp and v_exp of 8-bit pages."""
    i32 = torch.int32
    rows = _paged_dim("q", q, 3)
    dev = _paged_device("q", q)
    T, Hq, D = rows
    num_pages, Hkv, S, _ = _paged_dim("k_pages", pools[0], 4)
    B, max_pages = _paged_dim("block_table", block_table, 2)
    dt, pool = q.dtype, (num_pages, Hkv, S, D)
    if dt not in _PAGED_DTYPES:
        raise ValueError(f"q must be torch.float16 or torch.bfloat16, got {dt}")
    aq = _paged("q", q, dt, rows, dev)
    dims = _paged_dims_ref(B, Hq, Hkv, D, S, num_pages, max_pages, T, _PAGED_DTYPES[dt])
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _paged_workspace_of_one_call(dims.contents, q.device)
    (nbytes,) = _paged_dim("workspace", workspace, 1)
    pool_dtype = pool_dtype or dt
    more = [_paged(name, e, torch.int8, (num_pages, Hkv), dev) for name, e in zip(("k_exp", "v_exp"), exps)]
    status = getattr(lib(), fn)(
        dims, _int32("max_q_len", max_q_len), aq, _paged("k_pages", pools[0], pool_dtype, pool, dev),
        _paged("v_pages", pools[1], pool_dtype, pool, dev), *more,
        _paged("block_table", block_table, i32, (B, max_pages), dev), _paged("cu_q", cu_q, i32, (B + 1,), dev),
        _paged("kv_len", kv_len, i32, (B,), dev), scale, _paged("out", out, dt, rows, dev),
        _paged("workspace", workspace, torch.uint8, (nbytes,), dev), nbytes, _cuda_stream(dev))
    if status:
        _check(fn, status)
    return out


def gqa_paged_attn(q, k_pages, v_pages, block_table, cu_q, kv_len, scale: float, max_q_len: int, out=None,
                   workspace=None):
    """Attention of each request's new tokens over its pages: q [T,Hq,D] (request b owns rows
    cu_q[b]..cu_q[b+1]-1, the last of its kv_len[b] tokens), pages [num_pages,Hkv,S,D], block_table
    [B,max_pages]; every token attends to the tokens up to itself. max_q_len bounds the rows of a
    request. Rows of out outside the requests' are left as they were."""
    return _paged_attn("gqa_paged_attn", q, (k_pages, v_pages), None, (), block_table, cu_q, kv_len, scale, max_q_len, out, workspace)


def gqa_paged_attn_e4m3(q, k_pages, v_pages, k_exp, v_exp, block_table, cu_q, kv_len, scale: float, max_q_len: int, out=None,
                        workspace=None):
    """gqa_paged_attn over 8-bit pages: codes [num_pages,Hkv,S,D] uint8 and exponents [num_pages,Hkv] int8, a
    channel's value being value(code) * 2^exponent. The workspace is gqa_paged_attn's."""
    return _paged_attn("gqa_paged_attn_e4m3", q, (k_pages, v_pages), torch.uint8, (k_exp, v_exp), block_table, cu_q, kv_len, scale,
                       max_q_len, out, workspace)
