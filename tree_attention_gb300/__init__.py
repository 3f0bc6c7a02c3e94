"""Python binding of ``libtreeattn.so``, the sm_103a batched tree-attention
library (C ABI in ``include/tree_attn.h``).

The binding only marshals arguments: tensors are passed to the C entry points
as raw device pointers (by ctypes, or, for the calls of ``PagedCache`` and
``LatentCache``, by the extension module ``_binding``), every step of the computation runs in the
library's CUDA kernels, and there is no CPU fallback.  If the library has not been
built, importing works but every call raises ``RuntimeError``.

The operation is ``batch_tree_attn`` of the page "tree_attn.py"
(python/tvm/relax/frontend/nn/llm/tree_attn.py): ragged, multi-sequence GQA
attention over a causal prefix plus each q row's tree ancestors (DFS
``[enter, exit)`` intervals, ``_check_tree_order``), with optional inline
rotate-half RoPE (``_rope`` of the page "_kernel_common.py"), emitting the
output and the base-2 log-sum-exp.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Union

import torch

__all__ = [
    "TA_OK", "TA_ERR_INVALID_ARGUMENT", "TA_ERR_UNSUPPORTED", "TA_ERR_CUDA",
    "TA_ERR_DEVICE_TIMEOUT", "TreeAttnError", "Dims", "lib", "lib_path", "workspace_size",
    "tree_attn", "plan", "run", "device_status", "status_string", "mask_dense", "check_inputs",
    "TreeAttention", "PagedDims", "make_paged_dims", "paged_workspace_size", "tree_attn_paged",
    "MAX_CHUNKS", "split_workspace_size", "tree_attn_split", "merge_states", "last_cuda_error",
    "folds_rotation", "noalloc_device_status", "set_wait_hooks", "auto_split_chunks",
    "set_scheduler", "CacheDims", "Rope", "PagedCache", "cache_workspace_size", "LatentDims",
    "LatentCache", "latent_workspace_size", "reset_workspace", "ExpandedDims", "make_expanded_dims",
    "expanded_workspace_size", "tree_attn_expanded",
]

TA_OK = 0
TA_ERR_INVALID_ARGUMENT = 1
TA_ERR_UNSUPPORTED = 2
TA_ERR_CUDA = 3
TA_ERR_DEVICE_TIMEOUT = 4
TA_FP16 = 0
TA_BF16 = 1
MAX_CHUNKS = 16   # split-KV: most chunks per (sequence, q tile) pair

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libtreeattn.so")


class TreeAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = f"{what}: {status_string(status)} ({status})"
        if status == TA_ERR_CUDA:
            msg += f": {last_cuda_error()}"
        super().__init__(msg)
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("total_kv", ctypes.c_int32), ("total_tree", ctypes.c_int32),
                ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("rotary_mode", ctypes.c_int32)]


class PagedDims(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("total_tree", ctypes.c_int32), ("h_q", ctypes.c_int32),
                ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int32),
                ("nnz_pages", ctypes.c_int32)]


class CacheDims(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("h_q", ctypes.c_int32),
                ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int32),
                ("nnz_pages", ctypes.c_int32)]


class LatentDims(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("h_q", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int32),
                ("nnz_pages", ctypes.c_int32)]


class ExpandedDims(ctypes.Structure):
    _fields_ = [("batch_size", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("total_kv", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("turns", ctypes.c_uint64 * 64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(lib_path):
        raise RuntimeError(f"libtreeattn.so is not built ({lib_path}); run "
                           "tree_attention_gb300.build.build() or __graft_entry__.build()")
    L = ctypes.CDLL(lib_path)
    vp, i32p, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
    L.tree_attn_workspace_size.argtypes = [ctypes.POINTER(Dims)]
    L.tree_attn_workspace_size.restype = sz
    L.tree_attn.argtypes = [vp, i32p, vp, vp, i32p, i32p, i32p, i32p, vp, vp, ctypes.c_int32,
                            ctypes.c_float, ctypes.c_float, ctypes.c_float,
                            ctypes.POINTER(Dims), vp, sz, vp]
    L.tree_attn.restype = ctypes.c_int
    L.tree_attn_plan.argtypes = [i32p, i32p, i32p, i32p, i32p, ctypes.c_int32, ctypes.c_float,
                                 ctypes.c_float, ctypes.POINTER(Dims), vp, sz, vp]
    L.tree_attn_plan.restype = ctypes.c_int
    L.tree_attn_run.argtypes = [vp, vp, vp, i32p, i32p, i32p, i32p, i32p, vp, vp,
                                ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                ctypes.POINTER(Dims), vp, sz, vp]
    L.tree_attn_run.restype = ctypes.c_int
    L.tree_attn_noalloc.argtypes = [vp, i32p, vp, vp, i32p, i32p, i32p, i32p, vp, vp,
                                    ctypes.c_int32, ctypes.c_float, ctypes.c_float,
                                    ctypes.c_float, ctypes.POINTER(Dims), vp]
    L.tree_attn_noalloc.restype = ctypes.c_int
    L.tree_attn_device_status.argtypes = [vp, vp]
    L.tree_attn_device_status.restype = ctypes.c_int
    L.tree_attn_noalloc_device_status.argtypes = [vp]
    L.tree_attn_noalloc_device_status.restype = ctypes.c_int
    L.tree_attn_set_wait_hooks.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    L.tree_attn_set_wait_hooks.restype = ctypes.c_int
    L.tree_attn_last_cuda_error.argtypes = []
    L.tree_attn_last_cuda_error.restype = ctypes.c_char_p
    L.tree_attn_status_string.argtypes = [ctypes.c_int]
    L.tree_attn_status_string.restype = ctypes.c_char_p
    L.tree_attn_mask_dense.argtypes = [i32p, i32p, i32p, i32p, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_int32, vp, vp]
    L.tree_attn_mask_dense.restype = ctypes.c_int
    L.tree_attn_check_inputs.argtypes = [i32p, i32p, i32p, i32p, i32p, ctypes.POINTER(Dims)]
    L.tree_attn_check_inputs.restype = ctypes.c_int
    L.tree_attn_paged_workspace_size.argtypes = [ctypes.POINTER(PagedDims)]
    L.tree_attn_paged_workspace_size.restype = sz
    L.tree_attn_paged.argtypes = [vp, i32p, vp, i32p, i32p, i32p, i32p, i32p, vp, vp,
                                  ctypes.c_int32, ctypes.c_float, ctypes.POINTER(PagedDims), vp,
                                  sz, vp]
    L.tree_attn_paged.restype = ctypes.c_int
    L.tree_attn_split_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32]
    L.tree_attn_split_workspace_size.restype = sz
    L.tree_attn_set_scheduler.argtypes = [ctypes.c_int32]
    L.tree_attn_set_scheduler.restype = ctypes.c_int
    L.tree_attn_auto_split_chunks.argtypes = [ctypes.POINTER(Dims)]
    L.tree_attn_auto_split_chunks.restype = ctypes.c_int32
    L.tree_attn_split.argtypes = [vp, i32p, vp, vp, i32p, i32p, i32p, i32p, vp, vp,
                                  ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                  ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(Dims), vp, sz,
                                  vp]
    L.tree_attn_split.restype = ctypes.c_int
    L.tree_attn_merge_states.argtypes = [vp, vp, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                         ctypes.c_int, vp, vp, vp]
    L.tree_attn_merge_states.restype = ctypes.c_int
    i32, i64, f32, f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double
    cdims, rope = ctypes.POINTER(CacheDims), ctypes.POINTER(_RopeStruct)
    L.tree_attn_cache_workspace_size.argtypes = [cdims]
    L.tree_attn_cache_workspace_size.restype = sz
    L.tree_attn_rope_init.argtypes = [rope, i32, i32, f64, f64, f32, vp]
    L.tree_attn_rope_init.restype = ctypes.c_int
    L.tree_attn_append_paged.argtypes = [vp, i64, vp, i64, vp, i64, i32, i32p, i32p, vp, vp, f32,
                                         rope, vp, i32p, i32p, i32p, vp, cdims, vp, sz, vp]
    L.tree_attn_append_paged.restype = ctypes.c_int
    L.tree_attn_decode_paged.argtypes = [vp, vp, i32p, i32p, i32p, vp, vp, f32, cdims, vp, sz, vp]
    L.tree_attn_decode_paged.restype = ctypes.c_int
    L.tree_attn_compact_paged.argtypes = [vp, i32p, i32p, i32p, i32p, i32p, i32p, i32, i32p, i32p,
                                          i32p, i32p, i32p, cdims, vp, sz, vp]
    L.tree_attn_compact_paged.restype = ctypes.c_int
    L.tree_attn_copy_pages.argtypes = [vp, i32p, i32p, i32, cdims, vp, sz, vp]
    L.tree_attn_copy_pages.restype = ctypes.c_int
    ldims, edims = ctypes.POINTER(LatentDims), ctypes.POINTER(ExpandedDims)
    L.tree_attn_latent_workspace_size.argtypes = [ldims]
    L.tree_attn_latent_workspace_size.restype = sz
    L.tree_attn_append_latent.argtypes = [vp, i64, vp, i64, vp, i64, i64, i32, i32p, i32p, vp, f32,
                                          rope, vp, i32p, i32p, i32p, vp, i64, i64, vp, ldims, vp,
                                          sz, vp]
    L.tree_attn_append_latent.restype = ctypes.c_int
    L.tree_attn_decode_latent.argtypes = [vp, vp, i32p, i32p, i32p, vp, vp, f32, ldims, vp, sz, vp]
    L.tree_attn_decode_latent.restype = ctypes.c_int
    L.tree_attn_latent.argtypes = [vp, i32p, i32, vp, i32p, i32p, i32p, i32p, i32p, i32, vp, vp, f32,
                                   ldims, vp, sz, vp]
    L.tree_attn_latent.restype = ctypes.c_int
    L.tree_attn_compact_latent.argtypes = [vp, i32p, i32p, i32p, i32p, i32p, i32p, i32, i32p, i32p,
                                           i32p, i32p, i32p, ldims, vp, sz, vp]
    L.tree_attn_compact_latent.restype = ctypes.c_int
    L.tree_attn_copy_pages_latent.argtypes = [vp, i32p, i32p, i32, ldims, vp, sz, vp]
    L.tree_attn_copy_pages_latent.restype = ctypes.c_int
    L.tree_attn_expanded_workspace_size.argtypes = [edims]
    L.tree_attn_expanded_workspace_size.restype = sz
    L.tree_attn_expanded.argtypes = [vp, i64, i64, i32p, vp, i64, i64, vp, i64, vp, i64, i64, i32p, vp,
                                     vp, f32, edims, vp, sz, vp]
    L.tree_attn_expanded.restype = ctypes.c_int
    _lib = L
    return L


def status_string(status: int) -> str:
    try:
        return lib().tree_attn_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def last_cuda_error() -> str:
    """The CUDA error behind this thread's most recent TA_ERR_CUDA."""
    try:
        return lib().tree_attn_last_cuda_error().decode()
    except RuntimeError:
        return "unknown"


def folds_rotation(total_kv: int, device=None) -> bool:
    """Whether the one-call entry points fold the key rotation into the plan
    kernel (problems of at most 64 kv tokens per SM), i.e. launch two kernels
    instead of three under RoPE."""
    idx = torch.cuda.current_device() if device is None else device
    return total_kv <= 64 * torch.cuda.get_device_properties(idx).multi_processor_count


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float16:
        return TA_FP16
    if t == torch.bfloat16:
        return TA_BF16
    raise TypeError(f"unsupported dtype {t}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_dims(q: torch.Tensor, k: torch.Tensor, q_indptr: torch.Tensor,
              tree_order: torch.Tensor, rotary_mode: int = 0) -> Dims:
    return Dims(batch_size=q_indptr.numel() - 1, total_q=q.shape[0], total_kv=k.shape[0],
                total_tree=tree_order.shape[0], h_q=q.shape[1], h_kv=k.shape[1],
                head_dim=q.shape[2], dtype=_dtype_code(q.dtype), rotary_mode=int(rotary_mode))


def workspace_size(dims: Dims) -> int:
    return int(lib().tree_attn_workspace_size(ctypes.byref(dims)))


def auto_split_chunks(dims: Dims) -> int:
    """The split-KV chunk cap ``tree_attn`` uses for ``dims`` on the current
    device (1: no split; 0: invalid dims)."""
    return int(lib().tree_attn_auto_split_chunks(ctypes.byref(dims)))


def _check_dev(name: str, t: Optional[torch.Tensor], dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def tree_attn(q, q_indptr, k, v, kv_indptr, q_rope_position, mn_indptr, tree_order, out, lse,
              rotary_mode: int, rope_scale: float, rope_theta: float, sm_scale: float,
              workspace: torch.Tensor, stream=None) -> None:
    """Enqueue one batched tree attention on ``stream`` (default: torch's
    current stream).  All tensors are CUDA tensors with the layouts of
    ``include/tree_attn.h``; ``out`` and ``lse`` are written."""
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _check_dev(name, t, q.dtype)
    for name, t in (("q_indptr", q_indptr), ("kv_indptr", kv_indptr), ("mn_indptr", mn_indptr),
                    ("tree_order", tree_order), ("q_rope_position", q_rope_position)):
        _check_dev(name, t, torch.int32)
    _check_dev("lse", lse, torch.float32)
    _check_dev("workspace", workspace)
    dims = make_dims(q, k, q_indptr, tree_order, rotary_mode)
    st = lib().tree_attn(_ptr(q), _ptr(q_indptr), _ptr(k), _ptr(v), _ptr(kv_indptr),
                         _ptr(q_rope_position), _ptr(mn_indptr), _ptr(tree_order), _ptr(out),
                         _ptr(lse), int(rotary_mode), float(rope_scale), float(rope_theta),
                         float(sm_scale), ctypes.byref(dims), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn")


def tree_attn_noalloc(q, q_indptr, k, v, kv_indptr, q_rope_position, mn_indptr, tree_order,
                      out, lse, rotary_mode: int, rope_scale: float, rope_theta: float,
                      sm_scale: float, stream=None) -> None:
    """``tree_attn`` for callers that may not allocate device memory: the
    library's static 32 MiB device scratch array serves as the workspace.
    Calls share that array, so they must not overlap on the GPU."""
    dims = make_dims(q, k, q_indptr, tree_order, rotary_mode)
    st = lib().tree_attn_noalloc(_ptr(q), _ptr(q_indptr), _ptr(k), _ptr(v), _ptr(kv_indptr),
                                 _ptr(q_rope_position), _ptr(mn_indptr), _ptr(tree_order),
                                 _ptr(out), _ptr(lse), int(rotary_mode), float(rope_scale),
                                 float(rope_theta), float(sm_scale), ctypes.byref(dims),
                                 _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_noalloc")


def make_paged_dims(q: torch.Tensor, pages: torch.Tensor, q_indptr: torch.Tensor,
                    page_values: torch.Tensor, tree_order: torch.Tensor) -> PagedDims:
    return PagedDims(batch_size=q_indptr.numel() - 1, total_q=q.shape[0],
                     total_tree=tree_order.shape[0], h_q=q.shape[1], h_kv=pages.shape[2],
                     head_dim=q.shape[2], dtype=_dtype_code(q.dtype), num_pages=pages.shape[0],
                     nnz_pages=page_values.numel())


def paged_workspace_size(dims: PagedDims) -> int:
    return int(lib().tree_attn_paged_workspace_size(ctypes.byref(dims)))


def tree_attn_paged(q, q_indptr, pages, page_indptr, page_values, length_info, mn_indptr,
                    tree_order, out, lse, rotary_mode: int, sm_scale: float,
                    workspace: torch.Tensor, stream=None) -> None:
    """Enqueue tree attention over a paged KV cache (``pages [num_pages, 2,
    h_kv, 16, d]``, page table ``page_indptr``/``page_values``, last-page
    lengths ``length_info``); layouts as in ``include/tree_attn.h``."""
    for name, t in (("q", q), ("pages", pages), ("out", out)):
        _check_dev(name, t, q.dtype)
    for name, t in (("q_indptr", q_indptr), ("page_indptr", page_indptr),
                    ("page_values", page_values), ("length_info", length_info),
                    ("mn_indptr", mn_indptr), ("tree_order", tree_order)):
        _check_dev(name, t, torch.int32)
    _check_dev("lse", lse, torch.float32)
    _check_dev("workspace", workspace)
    if pages.dim() != 5 or pages.shape[1] != 2 or pages.shape[3] != 16:
        raise ValueError("pages must be [num_pages, 2, h_kv, 16, head_dim]")
    dims = make_paged_dims(q, pages, q_indptr, page_values, tree_order)
    st = lib().tree_attn_paged(_ptr(q), _ptr(q_indptr), _ptr(pages), _ptr(page_indptr),
                               _ptr(page_values), _ptr(length_info), _ptr(mn_indptr),
                               _ptr(tree_order), _ptr(out), _ptr(lse), int(rotary_mode),
                               float(sm_scale), ctypes.byref(dims), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_paged")


def split_workspace_size(dims: Dims, max_chunks: int) -> int:
    return int(lib().tree_attn_split_workspace_size(ctypes.byref(dims), int(max_chunks)))


def tree_attn_split(q, q_indptr, k, v, kv_indptr, q_rope_position, mn_indptr, tree_order, out,
                    lse, rotary_mode: int, rope_scale: float, rope_theta: float,
                    sm_scale: float, max_chunks: int, chunk_tiles: int,
                    workspace: torch.Tensor, stream=None) -> None:
    """``tree_attn`` with split-KV: pairs with many kv tiles are cut into up
    to ``max_chunks`` chunks of about ``chunk_tiles`` 128-column tiles (0: the
    plan picks the length), whose partial states a merge kernel combines.
    ``workspace`` holds ``split_workspace_size(dims, max_chunks)`` bytes."""
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _check_dev(name, t, q.dtype)
    for name, t in (("q_indptr", q_indptr), ("kv_indptr", kv_indptr), ("mn_indptr", mn_indptr),
                    ("tree_order", tree_order), ("q_rope_position", q_rope_position)):
        _check_dev(name, t, torch.int32)
    _check_dev("lse", lse, torch.float32)
    _check_dev("workspace", workspace)
    dims = make_dims(q, k, q_indptr, tree_order, rotary_mode)
    st = lib().tree_attn_split(_ptr(q), _ptr(q_indptr), _ptr(k), _ptr(v), _ptr(kv_indptr),
                               _ptr(q_rope_position), _ptr(mn_indptr), _ptr(tree_order),
                               _ptr(out), _ptr(lse), int(rotary_mode), float(rope_scale),
                               float(rope_theta), float(sm_scale), int(max_chunks),
                               int(chunk_tiles), ctypes.byref(dims), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_split")


def merge_states(parts: torch.Tensor, lses: torch.Tensor, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, stream=None):
    """Merge ``n`` attention states over disjoint kv sets: ``parts [n, ...,
    d]`` (fp16/bf16, normalised) and base-2 ``lses [n, ...]`` (float32) into
    ``out [..., d]`` and ``lse [...]`` (returned)."""
    _check_dev("parts", parts)
    _check_dev("lses", lses, torch.float32)
    if parts.dim() < 2 or tuple(lses.shape) != tuple(parts.shape[:-1]):
        raise ValueError("parts must be [n, ..., d] and lses [n, ...]")
    n, d = parts.shape[0], parts.shape[-1]
    rows = lses[0].numel() if n else 0
    if out is None:
        out = torch.empty(parts.shape[1:], dtype=parts.dtype, device=parts.device)
    if lse is None:
        lse = torch.empty(lses.shape[1:], dtype=torch.float32, device=parts.device)
    _check_dev("out", out, parts.dtype)
    _check_dev("lse", lse, torch.float32)
    st = lib().tree_attn_merge_states(_ptr(parts), _ptr(lses), int(n), int(rows), int(d),
                                      _dtype_code(parts.dtype), _ptr(out), _ptr(lse),
                                      _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_merge_states")
    return out, lse


def plan(q, q_indptr, k, kv_indptr, q_rope_position, mn_indptr, tree_order,
         rotary_mode: int, rope_scale: float, rope_theta: float, workspace: torch.Tensor,
         stream=None) -> None:
    """Enqueue the plan kernel (work items, tile classes, RoPE table); q and
    k are passed only for their shapes and dtype."""
    dims = make_dims(q, k, q_indptr, tree_order, rotary_mode)
    st = lib().tree_attn_plan(_ptr(q_indptr), _ptr(kv_indptr), _ptr(q_rope_position),
                              _ptr(mn_indptr), _ptr(tree_order), int(rotary_mode),
                              float(rope_scale), float(rope_theta), ctypes.byref(dims),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_plan")


def run(q, k, v, q_indptr, kv_indptr, q_rope_position, mn_indptr, tree_order, out, lse,
        rotary_mode: int, rope_scale: float, rope_theta: float, sm_scale: float,
        workspace: torch.Tensor, stream=None) -> None:
    """Enqueue the key rotation (RoPE) and the attention kernel on the plan
    held in ``workspace``."""
    dims = make_dims(q, k, q_indptr, tree_order, rotary_mode)
    st = lib().tree_attn_run(_ptr(q), _ptr(k), _ptr(v), _ptr(q_indptr), _ptr(kv_indptr),
                             _ptr(q_rope_position), _ptr(mn_indptr), _ptr(tree_order), _ptr(out),
                             _ptr(lse), int(rotary_mode), float(rope_scale), float(rope_theta),
                             float(sm_scale), ctypes.byref(dims), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_run")


def device_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status."""
    return int(lib().tree_attn_device_status(_ptr(workspace), _stream_ptr(stream)))


def noalloc_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status that
    ``tree_attn_noalloc`` calls left in the library's static scratch array."""
    return int(lib().tree_attn_noalloc_device_status(_stream_ptr(stream)))


def set_wait_hooks(wait_limit_ns: int = 0, stall: Union[bool, int] = False) -> None:
    """Test hook: the bounded-wait limit of later calls on this thread (0:
    the default) and whether their MMA threads first wait on a barrier that
    nothing arrives on (so that the wait runs out); ``-1 - i``: only that of the
    ``i``-th pair of SMs in ``LatentCache``'s attention."""
    st = lib().tree_attn_set_wait_hooks(int(wait_limit_ns), stall if stall < 0 else int(bool(stall)))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_set_wait_hooks")


def set_scheduler(mode: int) -> None:
    """Work scheduling of later calls' attention kernels on this thread: 0
    the atomic work queue, 1 cluster launch control (default)."""
    st = lib().tree_attn_set_scheduler(int(mode))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_set_scheduler")


def mask_dense(q_indptr, kv_indptr, mn_indptr, tree_order, total_q: int, max_kv: int,
               stream=None) -> torch.Tensor:
    """Dense visibility bytes ``[total_q, max_kv]`` from the device mask code."""
    vis = torch.zeros((max(total_q, 1), max(max_kv, 1)), dtype=torch.uint8,
                      device=q_indptr.device)
    st = lib().tree_attn_mask_dense(_ptr(q_indptr), _ptr(kv_indptr), _ptr(mn_indptr),
                                    _ptr(tree_order), q_indptr.numel() - 1, total_q, max_kv,
                                    _ptr(vis), _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_mask_dense")
    return vis[:total_q, :max_kv]


def check_inputs(q_indptr, kv_indptr, mn_indptr, tree_order, dims: Dims) -> int:
    """Host-side validation of host (CPU) int32 index arrays."""
    import numpy as np
    arrs = [np.ascontiguousarray(np.asarray(a, dtype=np.int32)) for a in
            (q_indptr, kv_indptr, mn_indptr, tree_order)]
    ptrs = [a.ctypes.data_as(ctypes.c_void_p) if a.size else None for a in arrs]
    return int(lib().tree_attn_check_inputs(ptrs[0], ptrs[1], ptrs[2], ptrs[3], None,
                                            ctypes.byref(dims)))


class TreeAttention:
    """Owns a workspace sized for one problem shape and runs the call.

    ``inputs`` is a dict of CUDA tensors with keys ``q, q_indptr, k, v,
    kv_indptr, q_rope_position (or None), mn_indptr, tree_order``."""

    def __init__(self, q, k, q_indptr, tree_order, rotary_mode: int, rope_scale: float,
                 rope_theta: float, sm_scale: float):
        self.dims = make_dims(q, k, q_indptr, tree_order, rotary_mode)
        n = workspace_size(self.dims)
        if n == 0:
            raise TreeAttnError(TA_ERR_UNSUPPORTED, "tree_attn_workspace_size")
        # zero-filled once: the library keeps its counters consistent afterwards
        self.workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
        self.rotary_mode, self.rope_scale = rotary_mode, rope_scale
        self.rope_theta, self.sm_scale = rope_theta, sm_scale

    def __call__(self, q, q_indptr, k, v, kv_indptr, q_rope_position, mn_indptr, tree_order,
                 out=None, lse=None, stream=None):
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        tree_attn(q, q_indptr, k, v, kv_indptr, q_rope_position, mn_indptr, tree_order, out,
                  lse, self.rotary_mode, self.rope_scale, self.rope_theta, self.sm_scale,
                  self.workspace, stream)
        return out, lse


def cache_workspace_size(dims: CacheDims) -> int:
    return int(lib().tree_attn_cache_workspace_size(ctypes.byref(dims)))


class Rope:
    """A rotation for ``PagedCache.append``: ``layout`` "half" (pairs j, j +
    rotary_dim / 2) or "interleaved" (pairs 2j, 2j + 1) on the first
    ``rotary_dim`` elements of a head, pair j turning by ``position * scale *
    theta ** (-2 j / rotary_dim)`` -- or ``position * scale * inv_freq[j]`` with
    a table of rotary_dim / 2 frequencies, for any rescaling of them for long
    contexts.  ``magnitude`` multiplies cos and sin."""

    LAYOUTS = {"half": 1, "interleaved": 2}

    def __init__(self, layout: str, rotary_dim: int, theta: float = 1e4, scale: float = 1.0,
                 magnitude: float = 1.0, inv_freq=None):
        if layout not in self.LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(self.LAYOUTS)}, got {layout!r}")
        table = None
        if inv_freq is not None:
            freq = [float(f) for f in inv_freq]
            if len(freq) != rotary_dim // 2:
                raise ValueError("inv_freq must have rotary_dim / 2 entries")
            table = (ctypes.c_double * len(freq))(*freq)
        self.struct = _RopeStruct()
        self.rotary_dim = int(rotary_dim)
        st = lib().tree_attn_rope_init(ctypes.byref(self.struct), self.LAYOUTS[layout],
                                       self.rotary_dim, float(theta), float(scale),
                                       float(magnitude), table)
        if st != TA_OK:
            raise TreeAttnError(st, "tree_attn_rope_init")
        self.address = ctypes.addressof(self.struct)


_binding_module = None


def _compiled():
    """The extension module with the compiled argument checks of PagedCache."""
    global _binding_module
    if _binding_module is None:
        lib()   # raises if it is not built
        import importlib
        try:
            _binding_module = importlib.import_module("tree_attention_gb300._binding")
        except ImportError as e:
            state = ("cannot be loaded" if os.path.exists(os.path.join(_PKG, "_binding.so"))
                     else "is not built")
            raise RuntimeError(f"_binding.so {state} ({e}); run tree_attention_gb300.build.build() "
                               "or __graft_entry__.build()") from e
    return _binding_module


def _bytes_of(workspace: torch.Tensor):
    """Where a workspace lies in its storage, which all tensors on it share."""
    storage = workspace.untyped_storage()
    start = workspace.data_ptr() - storage.data_ptr()
    return storage.__dict__, start, start + workspace.numel() * workspace.element_size()


def _claim(workspace: torch.Tensor, kind: str, used: bool = True) -> None:
    """Note that ``workspace`` is one of this kind of cache (if ``used``).  The two
    kinds keep what has to be zero between calls in different places, so memory that
    the other kind has had is refused, as whatever tensor it comes, until
    ``reset_workspace``."""
    notes, start, end = _bytes_of(workspace)
    claims = notes.setdefault("_tree_attn_claims", set())   # (start, end, kind)
    for a, b, other in claims:
        if other != kind and a < end and start < b:
            raise ValueError(f"workspace is one of the other kind of cache ({other}, not {kind})")
    if used:
        claims.add((start, end, kind))


def _as_stream(stream, device):
    """A stream object for a stream given as one or by address."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    address = int(getattr(stream, "cuda_stream", stream))
    # 0 and 1 are CUDA's names of the legacy default stream
    return (torch.cuda.ExternalStream(address, device=device) if address > 1
            else torch.cuda.default_stream(device))


def reset_workspace(workspace: torch.Tensor, stream=None) -> None:
    """Zero-fill a cache's workspace on ``stream`` (default: torch's current one),
    behind all calls on it, so that it may serve the other kind of cache.  Not while
    a graph is captured, whose replays would fill it again."""
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if workspace.is_cuda and torch.cuda.is_current_stream_capturing():
        raise ValueError("a workspace cannot be reset while a graph is captured")
    if stream is None:
        workspace.zero_()
    else:
        with torch.cuda.stream(_as_stream(stream, workspace.device)):
            workspace.zero_()
    notes, start, end = _bytes_of(workspace)
    claims = notes.get("_tree_attn_claims", set())
    for a, b, kind in list(claims):
        if a < end and start < b:
            claims.remove((a, b, kind))
            claims.update((x, y, kind) for x, y in ((a, start), (end, b)) if x < y)


class _Cache:
    """What ``PagedCache`` and ``LatentCache`` have in common: the pool, its page
    table and the workspace.  A subclass names its dims' size function and the
    extension module's calls."""

    def _attach(self, pages, page_indptr, page_values, length_info, dims, workspace):
        _check_dev("pages", pages)
        for name, t in (("page_indptr", page_indptr), ("page_values", page_values),
                        ("length_info", length_info)):
            _check_dev(name, t, torch.int32)
            if t.get_device() != pages.get_device():
                raise ValueError(f"{name} must be on the device of pages")
        if page_indptr.numel() != length_info.numel() + 1:
            raise ValueError("page_indptr must have one entry more than length_info")
        self.pages, self.page_indptr = pages, page_indptr
        self.page_values, self.length_info = page_values, length_info
        self.dtype, self.device = pages.dtype, pages.device
        self._dev = pages.get_device()
        self.batch_size = length_info.numel()
        self.dims = dims()
        self._binding = _compiled()
        with torch.cuda.device(self._dev):
            need = self._workspace_size(self.dims)
        if need == 0:
            raise TreeAttnError(TA_ERR_UNSUPPORTED, self._size_name)
        if workspace is not None:
            _check_dev("workspace", workspace)
            if workspace.get_device() != self._dev:
                raise ValueError("workspace must be on the device of pages")
            _claim(workspace, self._size_name, workspace.numel() * workspace.element_size() >= need)
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            # zero-filled once, before a call on any stream: the library keeps its
            # counters consistent afterwards.  While a graph is captured the filling
            # goes into it, as its replays may have other tensors in this memory
            # first, and is done at once too, for calls outside the graph
            workspace = torch.zeros(need, dtype=torch.uint8, device=self.device)
            if torch.cuda.is_current_stream_capturing():
                self._binding.zero_now(workspace)
            else:
                torch.cuda.current_stream(self._dev).synchronize()
            _claim(workspace, self._size_name)
        self.workspace = workspace
        # the addresses of these tensors are what the calls pass, so they stay
        self._held = (pages, page_indptr, page_values, length_info, workspace)
        self._handle = getattr(self._binding, self._prefix + "handle")(
            ctypes.addressof(self.dims), pages, page_indptr, page_values, length_info, workspace)
        self._compact = getattr(self._binding, self._prefix + "compact")
        self._copy_pages = getattr(self._binding, self._prefix + "copy_pages")

    def _empty(self, shape, dtype, stream):
        """A new output, from the pool of the stream that the call runs on."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(_as_stream(stream, self.device)):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def compact(self, mn_indptr, accept_indptr, accept_nodes, *, new_page_indptr=None,
                new_page_values=None, new_length_info=None, freed_pages=None, num_freed=None,
                stream=None):
        """Keep the accepted nodes (``accept_nodes`` ascending per sequence) of
        the trees that end the sequences (``mn_indptr``), moving their rows down
        behind the prefix.  Returns the new ``page_indptr, page_values,
        length_info`` (for ``with_table``), the freed pages and their number
        ``[1]``, all on the device."""
        i32, b, nnz = torch.int32, self.batch_size, self.page_values.numel()
        if new_page_indptr is None:
            new_page_indptr = self._empty(b + 1, i32, stream)
        if new_page_values is None:
            new_page_values = self._empty(nnz, i32, stream)
        if new_length_info is None:
            new_length_info = self._empty(b, i32, stream)
        if freed_pages is None:
            freed_pages = self._empty(nnz, i32, stream)
        if num_freed is None:
            num_freed = self._empty(1, i32, stream)
        st = self._compact(self._handle, mn_indptr, accept_indptr, accept_nodes, new_page_indptr,
                           new_page_values, new_length_info, freed_pages, num_freed, stream)
        if st != TA_OK:
            raise TreeAttnError(st, self._names[0])
        return new_page_indptr, new_page_values, new_length_info, freed_pages, num_freed

    def copy_pages(self, src_pages, dst_pages, stream=None) -> None:
        """``pages[dst_pages[i]] = pages[src_pages[i]]``; no destination may be
        another pair's source or destination."""
        st = self._copy_pages(self._handle, src_pages, dst_pages, stream)
        if st != TA_OK:
            raise TreeAttnError(st, self._names[1])

    def device_status(self, stream=None) -> int:
        """Synchronise the stream and return (and clear) the device status."""
        return device_status(self.workspace, stream)


class PagedCache(_Cache):
    """A paged KV cache and its page table, with the calls of a decoding loop
    on it (``include/tree_attn.h``, "Serving a paged KV cache").

    ``pages [num_pages, 2, h_kv, 16, d]`` and the int32 table ``page_indptr
    [B+1]``, ``page_values``, ``length_info [B]`` are CUDA tensors, held and not
    copied: their contents may change between calls.  ``h_q`` is the number of
    query heads.  The handle owns a workspace, so calls on it that may overlap
    on the GPU need handles of their own (``with_table(..., workspace=None)``).
    ``workspace`` takes another handle's, whatever that one's heads and pool,
    where it is large enough; where it is not, a new one is made.  Every call is
    asynchronous on ``stream`` (default: torch's current stream), and
    ``device_status`` reports inconsistent tables.  The handle may be dropped
    while its calls run, unless on a stream that is not one of torch's."""

    _prefix, _size_name = "", "tree_attn_cache_workspace_size"
    _names = ("tree_attn_compact_paged", "tree_attn_copy_pages")
    _workspace_size = staticmethod(cache_workspace_size)

    def __init__(self, pages, page_indptr, page_values, length_info, h_q: int, workspace=None):
        if pages.dim() != 5 or pages.shape[1] != 2 or pages.shape[3] != 16:
            raise ValueError("pages must be [num_pages, 2, h_kv, 16, head_dim]")
        self.h_q, self.h_kv, self.head_dim = int(h_q), pages.shape[2], pages.shape[4]
        self._attach(pages, page_indptr, page_values, length_info, lambda: CacheDims(
            batch_size=length_info.numel(), h_q=self.h_q, h_kv=self.h_kv, head_dim=self.head_dim,
            dtype=_dtype_code(pages.dtype), num_pages=pages.shape[0],
            nnz_pages=page_values.numel()), workspace)

    def with_table(self, page_indptr, page_values, length_info, workspace="same"):
        """A handle on the same pool with another page table (as ``compact``
        writes); it shares this handle's workspace where that is large enough,
        unless given another one (None: a new one)."""
        return PagedCache(self.pages, page_indptr, page_values, length_info, self.h_q,
                          self.workspace if isinstance(workspace, str) else workspace)

    def append(self, q, k, v, append_indptr, positions=None, *, rope: Optional[Rope] = None,
               q_weight=None, k_weight=None, norm_eps: float = 1e-6, q_out=None, stream=None):
        """Write new tokens' keys and values to the last rows of their
        sequences (``append_indptr [B+1]``) and return their queries, after the
        norm (where a weight is given) and the rotation (with ``rope``, at
        ``positions [tokens]``).  q, k, v are ``[tokens, heads, d]`` and may be
        views of one fused projection."""
        if rope is not None and positions is None:
            raise ValueError("rope needs positions")
        if q_out is None:
            q_out = self._empty((q.shape[0], self.h_q, self.head_dim), self.dtype, stream)
        st = self._binding.append(self._handle, q, k, v, append_indptr, positions,
                                  None if rope is None else rope.address, q_weight, k_weight,
                                  norm_eps, q_out, stream)
        if st != TA_OK:
            raise TreeAttnError(st, "tree_attn_append_paged")
        return q_out

    def decode(self, q, sm_scale: float, out=None, lse=None, stream=None):
        """Attention of one new token per sequence, ``q [B, h_q, d]``, over all
        its kv rows; returns ``out`` and the base-2 ``lse [B, h_q]``."""
        if out is None:
            out = self._empty((self.batch_size, self.h_q, self.head_dim), self.dtype, stream)
        if lse is None:
            lse = self._empty((self.batch_size, self.h_q), torch.float32, stream)
        st = self._binding.decode(self._handle, q, sm_scale, out, lse, stream)
        if st != TA_OK:
            raise TreeAttnError(st, "tree_attn_decode_paged")
        return out, lse


def latent_workspace_size(dims: LatentDims) -> int:
    return int(lib().tree_attn_latent_workspace_size(ctypes.byref(dims)))


class LatentCache(_Cache):
    """A paged latent cache and its page table, with the calls of a decoding loop
    on it (``include/tree_attn.h``, "Latent attention"): one row of ``rank``
    latent elements and a rotary key per token, which all heads share.

    ``pages [num_pages, 16, rank + rope_dim]``, the table and the workspace are
    held as ``PagedCache`` holds its own; everything said there holds here.  A
    workspace may be another ``LatentCache``'s, but a ``PagedCache``'s only after
    ``reset_workspace`` (and the other way round)."""

    _prefix, _size_name = "latent_", "tree_attn_latent_workspace_size"
    _names = ("tree_attn_compact_latent", "tree_attn_copy_pages_latent")
    _workspace_size = staticmethod(latent_workspace_size)

    def __init__(self, pages, page_indptr, page_values, length_info, h_q: int, rank: int,
                 workspace=None):
        if pages.dim() != 3 or pages.shape[1] != 16:
            raise ValueError("pages must be [num_pages, 16, rank + rope_dim]")
        self.h_q, self.rank, self.rope_dim = int(h_q), int(rank), pages.shape[2] - int(rank)
        self._attach(pages, page_indptr, page_values, length_info, lambda: LatentDims(
            batch_size=length_info.numel(), h_q=self.h_q, rank=self.rank, rope_dim=self.rope_dim,
            dtype=_dtype_code(pages.dtype), num_pages=pages.shape[0],
            nnz_pages=page_values.numel()), workspace)

    def with_table(self, page_indptr, page_values, length_info, workspace="same"):
        """A handle on the same pool with another page table (as ``compact``
        writes); it shares this handle's workspace where that is large enough,
        unless given another one (None: a new one)."""
        return LatentCache(self.pages, page_indptr, page_values, length_info, self.h_q, self.rank,
                           self.workspace if isinstance(workspace, str) else workspace)

    def append(self, latent, k_rope, append_indptr, positions=None, *, q_rope=None,
               rope: Optional[Rope] = None, weight=None, norm_eps: float = 1e-6, q_out=None,
               rows_out=None, stream=None):
        """Write new tokens' rows, ``latent [tokens, rank]`` after its norm (where
        ``weight`` is given) and ``k_rope [tokens, rope_dim]`` after the rotation
        (with ``rope``, at ``positions``), to the last rows of their sequences,
        and return the queries' rotary parts ``q_rope [tokens, h_q, rope_dim]``,
        rotated (None without any).  All of them, and ``q_out``, may be views with
        strides; ``rows_out [tokens, rank + rope_dim]`` takes the rows too."""
        if rope is not None and positions is None:
            raise ValueError("rope needs positions")
        if q_rope is None and q_out is not None:
            raise ValueError("q_out needs q_rope")
        if q_rope is not None and q_out is None:
            q_out = self._empty((latent.shape[0], self.h_q, self.rope_dim), self.dtype, stream)
        st = self._binding.latent_append(self._handle, latent, k_rope, q_rope, append_indptr,
                                         positions, None if rope is None else rope.address, weight,
                                         norm_eps, q_out, rows_out, stream)
        if st != TA_OK:
            raise TreeAttnError(st, "tree_attn_append_latent")
        return q_out

    def decode(self, q, sm_scale: float, out=None, lse=None, stream=None):
        """Absorbed attention of one new token per sequence, ``q [B, h_q, rank +
        rope_dim]``, over all its rows; returns ``out [B, h_q, rank]`` and the
        base-2 ``lse [B, h_q]``."""
        if out is None:
            out = self._empty((self.batch_size, self.h_q, self.rank), self.dtype, stream)
        if lse is None:
            lse = self._empty((self.batch_size, self.h_q), torch.float32, stream)
        st = self._binding.latent_decode(self._handle, q, sm_scale, out, lse, stream)
        if st != TA_OK:
            raise TreeAttnError(st, "tree_attn_decode_latent")
        return out, lse

    def tree_attn(self, q, q_indptr, mn_indptr, tree_order, sm_scale: float, out=None, lse=None,
                  stream=None):
        """Absorbed attention of draft trees' nodes, ``q [total_q, h_q, rank +
        rope_dim]``, over their sequences' rows, of which the last are the trees'
        (as ``tree_attn_paged``); returns ``out [total_q, h_q, rank]`` and ``lse``."""
        if out is None:
            out = self._empty((q.shape[0], self.h_q, self.rank), self.dtype, stream)
        if lse is None:
            lse = self._empty((q.shape[0], self.h_q), torch.float32, stream)
        st = self._binding.latent_tree(self._handle, q, q_indptr, mn_indptr, tree_order, sm_scale,
                                       out, lse, stream)
        if st != TA_OK:
            raise TreeAttnError(st, "tree_attn_latent")
        return out, lse


def make_expanded_dims(q: torch.Tensor, k: torch.Tensor, q_indptr: torch.Tensor) -> ExpandedDims:
    return ExpandedDims(batch_size=q_indptr.numel() - 1, total_q=q.shape[0], total_kv=k.shape[0],
                        heads=k.shape[1], head_dim=k.shape[2], rope_dim=q.shape[2] - k.shape[2],
                        dtype=_dtype_code(q.dtype))


def expanded_workspace_size(dims: ExpandedDims) -> int:
    return int(lib().tree_attn_expanded_workspace_size(ctypes.byref(dims)))


def _row_strides(name: str, t: torch.Tensor, dtype, shape):
    """Token and head strides of a tensor whose rows are contiguous."""
    if not t.is_cuda or t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {dtype} {shape} on a CUDA device, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if t.stride(-1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    # strides of dimensions of one say nothing
    head = t.stride(1) if t.dim() == 3 and shape[1] > 1 else shape[-1]
    return t.stride(0) if shape[0] > 1 else max(head, shape[-1]), head


def tree_attn_expanded(q, q_indptr, k, k_rope, v, kv_indptr, out, lse, sm_scale: float,
                       workspace: torch.Tensor, stream=None) -> None:
    """Enqueue causal attention in the expanded form of latent attention: ``q
    [total_q, heads, head_dim + rope_dim]`` (each sequence's last rows), ``k, v
    [total_kv, heads, head_dim]``, the shared rotary key ``k_rope [total_kv,
    rope_dim]``; all may be views with strides.  ``out [total_q, heads, head_dim]``
    and the base-2 ``lse`` are written; ``workspace`` holds
    ``expanded_workspace_size(dims)`` zero-filled bytes (``device_status``)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must have 3 dimensions")
    (nq, h, dq), (nk, _, d) = q.shape, k.shape
    dims = make_expanded_dims(q, k, q_indptr)
    qt, qh = _row_strides("q", q, q.dtype, (nq, h, dq))
    kt, kh = _row_strides("k", k, q.dtype, (nk, h, d))
    vt, vh = _row_strides("v", v, q.dtype, (nk, h, d))
    rt, _ = _row_strides("k_rope", k_rope, q.dtype, (nk, dq - d))
    for name, t, dtype, shape in (("out", out, q.dtype, (nq, h, d)),
                                  ("lse", lse, torch.float32, (nq, h)),
                                  ("kv_indptr", kv_indptr, torch.int32, (dims.batch_size + 1,)),
                                  ("q_indptr", q_indptr, torch.int32, (dims.batch_size + 1,))):
        _check_dev(name, t, dtype)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have the shape {shape}, got {tuple(t.shape)}")
    _check_dev("workspace", workspace)
    for name, t in (("k", k), ("v", v), ("k_rope", k_rope), ("out", out), ("lse", lse),
                    ("q_indptr", q_indptr), ("kv_indptr", kv_indptr), ("workspace", workspace)):
        if t.get_device() != q.get_device():
            raise ValueError(f"{name} must be on the device of q")
    if q.get_device() != torch.cuda.current_device():
        raise ValueError(f"q is on {q.device}, which is not the current device")
    st = lib().tree_attn_expanded(_ptr(q), qt, qh, _ptr(q_indptr), _ptr(k), kt, kh, _ptr(k_rope), rt,
                                  _ptr(v), vt, vh, _ptr(kv_indptr), _ptr(out), _ptr(lse),
                                  float(sm_scale), ctypes.byref(dims), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != TA_OK:
        raise TreeAttnError(st, "tree_attn_expanded")
