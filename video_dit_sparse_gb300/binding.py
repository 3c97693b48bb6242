"""ctypes binding of ``libsparse_attn.so`` (declared in include/sparse_attn.h).

Argument marshalling only: torch CUDA tensors are passed as raw device
pointers together with ``torch.cuda.current_stream()``.  Every step of the
path runs in the library's kernels; there is no CPU or PyTorch fallback, and
a missing library raises at import.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparse_attn.so")

SA_OK, SA_ERR_INVALID_ARG, SA_ERR_UNSUPPORTED, SA_ERR_CAPACITY = 0, 1, 2, 3
SA_ERR_BAD_INDEX, SA_ERR_TIMEOUT, SA_ERR_CUDA = 4, 5, 6
SA_DEVERR_ROW_PTR, SA_DEVERR_INDEX, SA_DEVERR_TIMEOUT, SA_DEVERR_CAPACITY = 1, 2, 4, 8
SA_SELECT_TOPK, SA_SELECT_THRESHOLD, SA_SELECT_MASS = 0, 1, 2
_MODES = {"topk": SA_SELECT_TOPK, "threshold": SA_SELECT_THRESHOLD, "mass": SA_SELECT_MASS}
SA_COLSTAT_MAX, SA_COLSTAT_SUM = 0, 1
_STATS = {"max": SA_COLSTAT_MAX, "sum": SA_COLSTAT_SUM}


class SparseAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {sparse_attn_status_string(status)} (status {status})")


class sa_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Nq", ctypes.c_int32),
                ("Nk", ctypes.c_int32), ("d", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int32)]


SA_OUT_BF16, SA_OUT_FP32 = 0, 1
_OUT = {torch.bfloat16: SA_OUT_BF16, torch.float32: SA_OUT_FP32}


class sa_select(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("topk", ctypes.c_int64),
                ("threshold", ctypes.c_double), ("mass", ctypes.c_double)]


class sa_voxel_grid(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("Hh", ctypes.c_int32), ("W", ctypes.c_int32),
                ("vt", ctypes.c_int32), ("vh", ctypes.c_int32), ("vw", ctypes.c_int32)]


class sa_strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


SA_ROPE_INTERLEAVED, SA_ROPE_HALF = 0, 1
_PAIRINGS = {"interleaved": SA_ROPE_INTERLEAVED, "half": SA_ROPE_HALF}


class sa_rope(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("axis_dim", ctypes.c_int32 * 3),
                ("pairing", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("theta", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double)), ("positions", ctypes.c_void_p),
                ("positions_b", ctypes.c_int64), ("grid", sa_voxel_grid),
                ("voxel_order", ctypes.c_int32), ("offset", ctypes.c_int64 * 3)]


class sa_masked(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("Nq", ctypes.c_int32), ("Nk", ctypes.c_int32), ("d", ctypes.c_int32),
                ("scale", ctypes.c_float), ("out_dtype", ctypes.c_int32), ("q", sa_strides),
                ("k", sa_strides), ("v", sa_strides), ("o", sa_strides), ("cap", ctypes.c_float),
                ("slopes", ctypes.c_void_p), ("causal", ctypes.c_int32), ("ndocs", ctypes.c_int32),
                ("docs_q", ctypes.c_void_p), ("docs_k", ctypes.c_void_p),
                ("prefix", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


class sa_evict(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("Nk", ctypes.c_int32),
                ("d", ctypes.c_int32), ("budget", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("lengths", ctypes.c_void_p), ("k", sa_strides),
                ("v", sa_strides), ("k_out", sa_strides), ("v_out", sa_strides)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
            "(nvcc, sm_103a). There is no fallback implementation.")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, vp = ctypes.POINTER, ctypes.c_int64, ctypes.c_void_p
    lib.sparse_attn_build_index_workspace_size.argtypes = [P(sa_problem)]
    lib.sparse_attn_build_index_workspace_size.restype = ctypes.c_size_t
    lib.sparse_attn_build_index.argtypes = [P(sa_problem), P(sa_select), vp, vp, vp, vp, i64,
                                            P(ctypes.c_int64), vp, ctypes.c_size_t, vp]
    lib.sparse_attn_build_index.restype = ctypes.c_int
    lib.sparse_attn_build_index_dense.argtypes = [P(sa_problem), P(sa_select), ctypes.c_int32, vp,
                                                  vp, vp, vp, vp, i64, P(ctypes.c_int64), vp,
                                                  ctypes.c_size_t, vp]
    lib.sparse_attn_build_index_dense.restype = ctypes.c_int
    lib.sparse_attn_forward.argtypes = [P(sa_problem), vp, vp, vp, vp, vp, i64, vp, vp, vp, vp]
    lib.sparse_attn_forward.restype = ctypes.c_int
    lib.sparse_attn_forward_delta.argtypes = [P(sa_problem), vp, vp, vp, vp, vp, i64, vp, vp,
                                              ctypes.c_float, vp, vp, vp]
    lib.sparse_attn_forward_delta.restype = ctypes.c_int
    lib.sparse_attn_layer_from_host.argtypes = [P(sa_problem), P(sa_select), vp, vp, vp, vp, vp, vp,
                                                vp, vp, vp, vp, vp, vp, i64, vp, ctypes.c_size_t,
                                                ctypes.c_int32, vp, vp, vp]
    lib.sparse_attn_layer_from_host.restype = ctypes.c_int
    lib.sparse_attn_index_from_bitmask.argtypes = [P(sa_problem), vp, vp, vp, i64, P(ctypes.c_int64), vp]
    lib.sparse_attn_index_from_bitmask.restype = ctypes.c_int
    lib.sparse_attn_index_from_block_mask.argtypes = [P(sa_problem), ctypes.c_int32, vp, vp, vp, i64,
                                                      P(ctypes.c_int64), vp]
    lib.sparse_attn_index_from_block_mask.restype = ctypes.c_int
    lib.sparse_attn_voxel_permute.argtypes = [P(sa_voxel_grid), ctypes.c_int32, ctypes.c_int32, vp,
                                              vp, ctypes.c_int32, vp]
    lib.sparse_attn_voxel_permute.restype = ctypes.c_int
    lib.sparse_attn_kv_window_append.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_int32, i64, vp, vp, vp, vp,
                                                 P(ctypes.c_int64), vp]
    lib.sparse_attn_kv_window_append.restype = ctypes.c_int
    ps = P(sa_strides)
    lib.sparse_attn_rope.argtypes = [P(sa_rope), ctypes.c_int32, vp, ps, vp, ps, ctypes.c_int32, vp,
                                     ps, vp, ps, vp]
    lib.sparse_attn_rope.restype = ctypes.c_int
    lib.sparse_attn_forward_masked_workspace_size.argtypes = [P(sa_masked)]
    lib.sparse_attn_forward_masked_workspace_size.restype = ctypes.c_size_t
    lib.sparse_attn_forward_masked.argtypes = [P(sa_masked), vp, vp, vp, vp, vp, vp, vp,
                                               ctypes.c_size_t, vp]
    lib.sparse_attn_forward_masked.restype = ctypes.c_int
    lib.sparse_attn_cache_weights.argtypes = [P(sa_masked), vp, vp, vp, vp, vp, ctypes.c_float, vp, vp]
    lib.sparse_attn_cache_weights.restype = ctypes.c_int
    lib.sparse_attn_cache_evict.argtypes = [P(sa_evict), vp, vp, vp, vp, vp, vp, vp, vp]
    lib.sparse_attn_cache_evict.restype = ctypes.c_int
    lib.sparse_attn_validate_index.argtypes = [P(sa_problem), vp, vp, i64, vp, vp]
    lib.sparse_attn_validate_index.restype = ctypes.c_int
    lib.sparse_attn_status_string.argtypes = [ctypes.c_int]
    lib.sparse_attn_status_string.restype = ctypes.c_char_p
    lib.sparse_attn_version.argtypes = []
    lib.sparse_attn_version.restype = ctypes.c_int32
    return lib


lib = _load()


def sparse_attn_status_string(status: int) -> str:
    return lib.sparse_attn_status_string(int(status)).decode()


def sparse_attn_version() -> int:
    return int(lib.sparse_attn_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def problem(q: torch.Tensor, k: torch.Tensor, group_size: int, scale: float | None = None,
            out_dtype=torch.bfloat16):
    """sa_problem for bf16 [B,H,N,d] tensors."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, N, d]")
    B, H, Nq, d = q.shape
    if k.shape[0] != B or k.shape[1] != H or k.shape[3] != d:
        raise ValueError("k must be [B, H, Nk, d] with q's B, H and d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out_dtype not in _OUT:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    return sa_problem(B, H, Nq, k.shape[2], d, group_size, scale, _OUT[out_dtype])


def _check(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dtype}")


def sparse_attn_build_index_workspace_size(p: sa_problem) -> int:
    return int(lib.sparse_attn_build_index_workspace_size(ctypes.byref(p)))


def _build(q, k, mode, topk, threshold, mass, group_size, scale, col_capacity, workspace,
           stream, sync_nnz, stat=None, lse=None):
    _check(q, torch.bfloat16, "q")
    _check(k, torch.bfloat16, "k")
    p = problem(q, k, group_size, scale)
    G = -(-p.Nq // group_size)
    rows = p.B * p.H * G
    m = _MODES.get(mode, mode)
    sel = sa_select(m, int(topk), float(threshold), float(mass))
    dev = q.device
    row_ptr = torch.empty(rows + 1, dtype=torch.int64, device=dev)
    if col_capacity is None:
        col_capacity = rows * (min(max(int(topk), 1), p.Nk) if m == SA_SELECT_TOPK else p.Nk)
    col_idx = torch.empty(max(col_capacity, 1), dtype=torch.int32, device=dev)
    ws_bytes = sparse_attn_build_index_workspace_size(p)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if sync_nnz is None:
        sync_nnz = True
    nnz = ctypes.c_int64(0)
    nnz_ref = ctypes.byref(nnz) if sync_nnz else None
    if stat is None:
        st = lib.sparse_attn_build_index(ctypes.byref(p), ctypes.byref(sel), _ptr(q), _ptr(k),
                                         _ptr(row_ptr), _ptr(col_idx), int(col_capacity), nnz_ref,
                                         _ptr(workspace), workspace.numel(), _stream(stream))
        where = "sparse_attn_build_index"
    else:
        _check(lse, torch.float32, "lse")
        st = lib.sparse_attn_build_index_dense(ctypes.byref(p), ctypes.byref(sel),
                                               _STATS.get(stat, stat), _ptr(q), _ptr(k), _ptr(lse),
                                               _ptr(row_ptr), _ptr(col_idx), int(col_capacity),
                                               nnz_ref, _ptr(workspace), workspace.numel(),
                                               _stream(stream))
        where = "sparse_attn_build_index_dense"
    if st != SA_OK:
        raise SparseAttnError(st, where)
    n = nnz.value if sync_nnz else rows * min(max(int(topk), 1), p.Nk)
    return row_ptr, col_idx[:n], n


def sparse_attn_build_index(q: torch.Tensor, k: torch.Tensor, mode="topk", *, topk: int = 0,
                            threshold: float = 0.0, mass: float = 0.99, group_size: int = 128,
                            scale: float | None = None, col_capacity: int | None = None,
                            workspace: torch.Tensor | None = None, stream=None,
                            sync_nnz: bool | None = None):
    """Builds CSR key lists from mean-query scores; returns (row_ptr int64,
    col_idx int32, nnz).

    By default the call synchronises and raises on any device-side error
    (capacity, timeout).  ``sync_nnz=False`` keeps a TOPK call fully
    asynchronous (nnz is then known up front).  For THRESHOLD/MASS col_idx is
    allocated for the worst case (every key) unless col_capacity is given;
    col_idx is returned trimmed to nnz (a view).
    """
    return _build(q, k, mode, topk, threshold, mass, group_size, scale, col_capacity, workspace,
                  stream, sync_nnz)


def sparse_attn_build_index_dense(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor,
                                  stat="max", mode="threshold", *, topk: int = 0,
                                  threshold: float = 0.0, mass: float = 0.99,
                                  group_size: int = 128, scale: float | None = None,
                                  col_capacity: int | None = None,
                                  workspace: torch.Tensor | None = None, stream=None,
                                  sync_nnz: bool | None = None):
    """Key lists from a dense step's attention probabilities (column max or
    column sum over each group of exp(scale q.k - lse)); `lse` fp32
    [B,H,Nq] as the dense forward writes it.  THRESHOLD compares the
    statistic itself with `threshold` (the cached mask: stat "max",
    threshold 0.5/Nk).  Returns (row_ptr, col_idx, nnz) like
    sparse_attn_build_index."""
    return _build(q, k, mode, topk, threshold, mass, group_size, scale, col_capacity, workspace,
                  stream, sync_nnz, stat=stat, lse=lse)


def _fwd_common(q, k, v, row_ptr, col_idx, group_size, scale, nnz, out, out_dtype):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, torch.bfloat16, n)
    if (row_ptr is None) != (col_idx is None):
        raise ValueError("row_ptr and col_idx are both given or both None (dense)")
    if row_ptr is not None:
        _check(row_ptr, torch.int64, "row_ptr")
        _check(col_idx, torch.int32, "col_idx")
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    if out is not None:
        _check(out, out.dtype, "out")
        out_dtype = out.dtype
    p = problem(q, k, group_size, scale, out_dtype)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if row_ptr is None:
        return p, out, None, None, 0
    if nnz is None:
        nnz = col_idx.numel()
    return p, out, _ptr(row_ptr), (_ptr(col_idx) if col_idx.numel() else None), int(nnz)


def sparse_attn_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        row_ptr: torch.Tensor | None, col_idx: torch.Tensor | None, *,
                        group_size: int = 128, scale: float | None = None,
                        nnz: int | None = None, out: torch.Tensor | None = None,
                        out_dtype=torch.bfloat16, lse: torch.Tensor | bool = True,
                        status: torch.Tensor | None = None, stream=None):
    """Column-sparse attention; returns (o [B,H,Nq,d] in out_dtype (bf16 or
    fp32; taken from `out` if given), lse fp32 [B,H,Nq] or None).
    row_ptr = col_idx = None: dense attention (every key kept)."""
    p, out, rp, ci, nnz = _fwd_common(q, k, v, row_ptr, col_idx, group_size, scale, nnz, out,
                                      out_dtype)
    if lse is True:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    elif lse is False:
        lse = None
    st = lib.sparse_attn_forward(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), rp, ci, nnz,
                                 _ptr(out), _ptr(lse), _ptr(status), _stream(stream))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_forward")
    return out, lse


def sparse_attn_forward_delta(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              row_ptr: torch.Tensor | None, col_idx: torch.Tensor | None,
                              lse_ref: torch.Tensor, *, base: torch.Tensor | None = None,
                              sign: float = 1.0, group_size: int = 128,
                              scale: float | None = None, nnz: int | None = None,
                              out: torch.Tensor | None = None, out_dtype=torch.float32,
                              status: torch.Tensor | None = None, stream=None):
    """Sparse delta: o = base + sign * sum over kept j of
    exp(scale q.k_j - lse_ref) v_j (fp32 base, fp32 output by default;
    out=base updates the cache in place)."""
    _check(lse_ref, torch.float32, "lse_ref")
    if base is not None:
        _check(base, torch.float32, "base")
    p, out, rp, ci, nnz = _fwd_common(q, k, v, row_ptr, col_idx, group_size, scale, nnz, out,
                                      out_dtype)
    st = lib.sparse_attn_forward_delta(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), rp, ci, nnz,
                                       _ptr(lse_ref), _ptr(base), float(sign), _ptr(out),
                                       _ptr(status), _stream(stream))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_forward_delta")
    return out


def sparse_attn_validate_index(row_ptr: torch.Tensor, col_idx: torch.Tensor, *, B: int, H: int,
                               Nq: int, Nk: int, d: int = 128, group_size: int = 128,
                               status: torch.Tensor | None = None, stream=None) -> int:
    """Returns SA_OK or SA_ERR_BAD_INDEX (synchronises)."""
    _check(row_ptr, torch.int64, "row_ptr")
    _check(col_idx, torch.int32, "col_idx")
    p = sa_problem(B, H, Nq, Nk, d, group_size, 1.0 / math.sqrt(d), SA_OUT_BF16)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=row_ptr.device)
    st = lib.sparse_attn_validate_index(ctypes.byref(p), _ptr(row_ptr),
                                        _ptr(col_idx) if col_idx.numel() else None,
                                        col_idx.numel(), _ptr(status), _stream(stream))
    if st not in (SA_OK, SA_ERR_BAD_INDEX):
        raise SparseAttnError(st, "sparse_attn_validate_index")
    return st


def _from_mask(mask, B, H, Nq, Nk, d, group_size, block_k, col_capacity, stream):
    p = sa_problem(B, H, Nq, Nk, d, group_size, 1.0 / math.sqrt(d), SA_OUT_BF16)
    G = -(-Nq // group_size)
    rows = B * H * G
    dev = mask.device
    row_ptr = torch.empty(rows + 1, dtype=torch.int64, device=dev)
    cap = rows * Nk if col_capacity is None else int(col_capacity)
    col_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    nnz = ctypes.c_int64(0)
    if block_k is None:
        st = lib.sparse_attn_index_from_bitmask(ctypes.byref(p), _ptr(mask), _ptr(row_ptr),
                                                _ptr(col_idx), cap, ctypes.byref(nnz), _stream(stream))
        where = "sparse_attn_index_from_bitmask"
    else:
        st = lib.sparse_attn_index_from_block_mask(ctypes.byref(p), int(block_k), _ptr(mask),
                                                   _ptr(row_ptr), _ptr(col_idx), cap,
                                                   ctypes.byref(nnz), _stream(stream))
        where = "sparse_attn_index_from_block_mask"
    if st != SA_OK:
        raise SparseAttnError(st, where)
    return row_ptr, col_idx[:nnz.value], nnz.value


def sparse_attn_index_from_bitmask(mask_words: torch.Tensor, *, B: int, H: int, Nq: int, Nk: int,
                                   d: int = 128, group_size: int = 128,
                                   col_capacity: int | None = None, stream=None):
    """uint32 words [B*H*G, ceil(Nk/32)] (torch.int32 storage), key j = bit j%32
    of word j//32 -> (row_ptr, col_idx, nnz).  Synchronises."""
    _check(mask_words, torch.int32, "mask_words")
    return _from_mask(mask_words, B, H, Nq, Nk, d, group_size, None, col_capacity, stream)


def sparse_attn_index_from_block_mask(block_mask: torch.Tensor, block_k: int, *, B: int, H: int,
                                      Nq: int, Nk: int, d: int = 128, group_size: int = 128,
                                      col_capacity: int | None = None, stream=None):
    """uint8 [B*H*G, ceil(Nk/block_k)] (non-zero = keep the key block) ->
    (row_ptr, col_idx, nnz).  Synchronises."""
    _check(block_mask, torch.uint8, "block_mask")
    return _from_mask(block_mask, B, H, Nq, Nk, d, group_size, block_k, col_capacity, stream)


def sparse_attn_voxel_permute(x: torch.Tensor, grid, voxel, *, inverse: bool = False,
                              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x bf16 [B, H, N, d] (N = T*Hh*W) -> the same tokens in voxel order
    (or back to raster order when inverse)."""
    _check(x, torch.bfloat16, "x")
    if x.dim() != 4:
        raise ValueError("x must be [B, H, N, d]")
    B, H, N, d = x.shape
    g = sa_voxel_grid(*grid, *voxel)
    if out is None:
        out = torch.empty_like(x)
    _check(out, torch.bfloat16, "out")
    st = lib.sparse_attn_voxel_permute(ctypes.byref(g), B * H, d, _ptr(x), _ptr(out),
                                       1 if inverse else 0, _stream(stream))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_voxel_permute")
    return out


def sparse_attn_kv_window_append(cache_k: torch.Tensor, cache_v: torch.Tensor,
                                 new_k: torch.Tensor, new_v: torch.Tensor, chunks_before: int, *,
                                 stream=None) -> int:
    """Appends one chunk ([B, H, L, d]) to the rolling caches ([B, H, S*L, d],
    slot 0 = sink) in place; returns the number of valid key tokens."""
    for t, n in ((cache_k, "cache_k"), (cache_v, "cache_v"), (new_k, "new_k"), (new_v, "new_v")):
        _check(t, torch.bfloat16, n)
    B, H, SL, d = cache_k.shape
    L = new_k.shape[2]
    if cache_v.shape != cache_k.shape or new_v.shape != new_k.shape or SL % L:
        raise ValueError("caches must be [B, H, S*L, d] and chunks [B, H, L, d]")
    valid = ctypes.c_int64(0)
    st = lib.sparse_attn_kv_window_append(B * H, d, L, SL // L, int(chunks_before), _ptr(cache_k),
                                          _ptr(cache_v), _ptr(new_k), _ptr(new_v),
                                          ctypes.byref(valid), _stream(stream))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_kv_window_append")
    return int(valid.value)


# ------------------------------------------------ operators around the attention path
#
# A call on a small problem takes the GPU a few microseconds, so what Python does per call counts:
# problems are packed in one go (the structures above say what their fields are) and passed as bytes.

_MASKED = struct.Struct("@6ifi12qfP2i4P")
_EVICT = struct.Struct("@7iP12q")
_ROPE = struct.Struct("@10id2Pq6ii3q")
assert _MASKED.size == ctypes.sizeof(sa_masked) and _EVICT.size == ctypes.sizeof(sa_evict)
assert _ROPE.size == ctypes.sizeof(sa_rope)
_STRIDES = struct.Struct("@3q")
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32
_empty, _empty_like = torch.empty, torch.empty_like
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _by_bytes(name, argtypes, restype=ctypes.c_int):
    f = lib[name]  # its own function object: the declared prototype stays as it is
    f.argtypes, f.restype = argtypes, restype
    return f


_vp, _cp = ctypes.c_void_p, ctypes.c_char_p
_c_rope = _by_bytes("sparse_attn_rope", [_cp, ctypes.c_int32, _vp, _cp, _vp, _cp, ctypes.c_int32, _vp, _cp, _vp, _cp, _vp])
_c_masked = _by_bytes("sparse_attn_forward_masked", [_cp] + [_vp] * 7 + [ctypes.c_size_t, _vp])
_c_masked_ws = _by_bytes("sparse_attn_forward_masked_workspace_size", [_cp], ctypes.c_size_t)
_c_weights = _by_bytes("sparse_attn_cache_weights", [_cp] + [_vp] * 5 + [ctypes.c_float, _vp, _vp])
_c_evict = _by_bytes("sparse_attn_cache_evict", [_cp] + [_vp] * 8)


def _view(t: torch.Tensor, dtype, name: str, dev: int):
    """The strides of a view [B, H, N, d] with a contiguous d on CUDA device `dev`."""
    if t.dtype is not dtype or t.dim() != 4 or t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor [B, H, N, d] of {dtype}, on the first tensor's device")
    sb, sh, sn, sd = t.stride()
    if sd != 1 and t.shape[3] != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return sb, sh, sn


def _flat(t, dtype, name, dev, shape=None) -> int:
    """The address of a contiguous tensor on device `dev` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {dtype} on the first tensor's device")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t.data_ptr()


def _elsewhere(dev: int, stream, call, *args, **options):
    """The call with the tensors' device current and, when one is given, on `stream`: what the call
    makes and fills is made there, and its results are not reused while the caller's stream may
    still read them."""
    if stream is None:
        with torch.cuda.device(dev):
            return call(*args, **options)
    if stream.device.index != dev:
        raise ValueError("stream must be on the first tensor's device")
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        made = call(*args, **options)
        for t in made if isinstance(made, tuple) else (made,):
            if t is not None:
                t.record_stream(here)
    return made


def sparse_attn_rope(q: torch.Tensor, k: torch.Tensor | None = None, *, axes=(44, 42, 42),
                     theta: float = 10000.0, inv_freq=None, pairing: str = "interleaved",
                     grid=None, voxel=None, offset=(0, 0, 0), positions: torch.Tensor | None = None,
                     inverse: bool = False, out=None, stream=None):
    """Rotary positions along up to three axes of q (and k, in the same launch): [B, H, N, d] bf16
    or fp32 views; returns the rotated q, or (q, k) when k is given.

    axes: rotated elements per axis.  positions int32 [N, A] or [B, N, A]; or grid (T, H, W) with
    N = T*H*W, tokens in raster order, or in sparse_attn_voxel_permute's when `voxel` is given, plus
    `offset`.  inv_freq: r/2 frequencies (radians per position) instead of theta's.  inverse rotates
    back, which is also the gradient.  out: the output (or a pair of them); it may be the input."""
    dtype, dev = q.dtype, q.get_device()
    if dev >= 0 and (stream is not None or dev != _current_device()):
        return _elsewhere(dev, stream, sparse_attn_rope, q, k, axes=axes, theta=theta, inv_freq=inv_freq,
                          pairing=pairing, grid=grid, voxel=voxel, offset=offset, positions=positions,
                          inverse=inverse, out=out)
    if dtype not in _OUT:
        raise ValueError("q must be bfloat16 or float32")
    qs = _view(q, dtype, "q", dev)
    B, H, N, d = q.shape
    oq, ok = out if isinstance(out, (tuple, list)) else (out, None)
    if k is not None:
        ks = _STRIDES.pack(*_view(k, dtype, "k", dev))
        if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
            raise ValueError("k must be [B, Hk, N, d] with q's B, N and d")
    elif ok is not None:
        raise ValueError("an output for k without k")
    na = len(axes)
    if not 1 <= na <= 3:
        raise ValueError("one to three axes")
    if pairing not in _PAIRINGS:
        raise ValueError("pairing must be 'interleaved' or 'half'")
    freq = 0
    if inv_freq is not None:
        f = [float(x) for x in inv_freq]
        if len(f) != sum(axes) // 2:
            raise ValueError("inv_freq must have one value per rotated pair")
        host = (ctypes.c_double * len(f))(*f)
        freq = ctypes.addressof(host)
    if (positions is None) == (grid is None):
        raise ValueError("positions or grid, and not both")
    pos = pos_b = 0
    cells, order = (0, 0, 0, 0, 0, 0), 0
    if positions is not None:
        if voxel is not None or any(offset):
            raise ValueError("voxel and offset go with grid")
        shared = positions.dim() == 2
        pos = _flat(positions, _i32, "positions", dev, (N, na) if shared else (B, N, na))
        pos_b = 0 if shared else N * na
    else:
        order = 0 if voxel is None else 1
        cells = (*grid, *(voxel or (0, 0, 0)))
    p = _ROPE.pack(B, N, d, na, *axes, *(0,) * (3 - na), _PAIRINGS[pairing], _OUT[dtype],
                   1 if inverse else 0, theta, freq, pos, pos_b, *cells, order, *offset)
    y = _empty_like(q) if oq is None else oq
    if y.shape != q.shape:
        raise ValueError("out must have q's shape")
    ys = _STRIDES.pack(*_view(y, dtype, "out", dev))
    z = None
    if k is None:
        st = _c_rope(p, H, q.data_ptr(), _STRIDES.pack(*qs), y.data_ptr(), ys, 0, None, None, None, None,
                     _current_stream(dev))
    else:
        z = _empty_like(k) if ok is None else ok
        if z.shape != k.shape:
            raise ValueError("out of k must have k's shape")
        st = _c_rope(p, H, q.data_ptr(), _STRIDES.pack(*qs), y.data_ptr(), ys, k.shape[1], k.data_ptr(), ks,
                     z.data_ptr(), _STRIDES.pack(*_view(z, dtype, "out of k", dev)),
                     _current_stream(dev))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_rope")
    return y if k is None else (y, z)


def _mask_fields(q, k, dev, slopes, docs_q, docs_k, prefix, lengths):
    """The mask's tables: (number of documents, their addresses, tensors to keep until the launch)."""
    B, H, _, d = q.shape
    kb, kh, _, kd = k.shape
    if kb != B or kd != d or not kh or H % kh:
        raise ValueError("k must be [B, Hk, Nk, d] with q's B and d, and H a multiple of Hk")
    slopes = 0 if slopes is None else _flat(slopes, _f32, "slopes", dev, (H,))
    n, made = 0, ()
    if docs_q is None:
        if docs_k is not None or prefix is not None:
            raise ValueError("docs_q and docs_k come together, prefix with them")
        dq = dk = px = 0
    else:
        if docs_k is None:
            raise ValueError("docs_q and docs_k come together, prefix with them")
        n = docs_q.shape[-1] - 1
        if n < 1:
            raise ValueError("docs_q must hold the bounds of at least one document")
        if docs_q.dim() == 1 and B > 1:
            docs_q, docs_k = (t.expand(B, n + 1).contiguous() for t in (docs_q, docs_k))
            prefix = None if prefix is None else prefix.expand(B, n).contiguous()
            made = (docs_q, docs_k, prefix)
        one = docs_q.dim() == 1
        dq = _flat(docs_q, _i32, "docs_q", dev, (n + 1,) if one else (B, n + 1))
        dk = _flat(docs_k, _i32, "docs_k", dev, (n + 1,) if one else (B, n + 1))
        px = _flat(prefix, _i32, "prefix", dev, (n,) if one else (B, n))
    lengths = 0 if lengths is None else _flat(lengths, _i32, "lengths", dev, (B,))
    return n, slopes, dq, dk, px, lengths, made


def sparse_attn_forward_masked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                               scale: float | None = None, cap: float = 0.0,
                               slopes: torch.Tensor | None = None, causal: int = 0,
                               docs_q: torch.Tensor | None = None,
                               docs_k: torch.Tensor | None = None,
                               prefix: torch.Tensor | None = None,
                               lengths: torch.Tensor | None = None,
                               out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                               lse: torch.Tensor | bool = True,
                               workspace: torch.Tensor | None = None,
                               status: torch.Tensor | None = None, stream=None):
    """Attention with masks, capped scores and a distance bias; bf16 views q [B, H, Nq, d],
    k and v [B, Hk, Nk, d] (H a multiple of Hk).  Returns (o [B, H, Nq, d], lse fp32 [B, H, Nq] or
    None).

    s = cap tanh(scale q.k / cap) - slopes[h] |p - c| over the keys a row sees: its document's
    (docs_q, docs_k int32 [n+1] or [B, n+1]; or the first lengths[b] keys), up to the end of its
    frame when `causal` (tokens per frame, 1: per token), and the document's first `prefix` keys.  A
    document's rows are its last positions, so one new token over a cache is Nq = 1 with lengths."""
    dev = q.get_device()
    if dev >= 0 and (stream is not None or dev != _current_device()):
        return _elsewhere(dev, stream, sparse_attn_forward_masked, q, k, v, scale=scale, cap=cap,
                          slopes=slopes, causal=causal, docs_q=docs_q, docs_k=docs_k, prefix=prefix,
                          lengths=lengths, out=out, out_dtype=out_dtype, lse=lse, workspace=workspace,
                          status=status)
    qs, ks = _view(q, _bf16, "q", dev), _view(k, _bf16, "k", dev)
    vs = _view(v, _bf16, "v", dev)
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    n, sl, dq, dk, px, lens, made = _mask_fields(q, k, dev, slopes, docs_q, docs_k, prefix, lengths)
    B, H, Nq, d = shape = q.shape
    if out is None:
        out = _empty_like(q) if out_dtype is q.dtype else _empty_like(q, dtype=out_dtype)
    elif out.shape != shape:
        raise ValueError("out must have q's shape")
    if out.dtype not in _OUT:
        raise ValueError("out must be bfloat16 or float32")
    if lse is True:
        lse = _empty(shape[:3], dtype=_f32, device=q.device)
    elif lse is False:
        lse = None
    p = _MASKED.pack(B, H, k.shape[1], Nq, k.shape[2], d, 1.0 / math.sqrt(d) if scale is None else scale,
                     _OUT[out.dtype], *qs, *ks, *vs, *_view(out, out.dtype, "out", dev), cap, sl, causal, n,
                     dq, dk, px, lens)
    need = _c_masked_ws(p)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = _c_masked(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                   _flat(lse, _f32, "lse", dev, shape[:3]), 0 if status is None else _flat(status, _i32, "status", dev),
                   _flat(workspace, torch.uint8, "workspace", dev),
                   0 if workspace is None else workspace.numel(),
                   _current_stream(dev))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_forward_masked")
    return out, lse


def sparse_attn_cache_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor,
                              weights: torch.Tensor | None = None, *, decay: float = 1.0,
                              scale: float | None = None, cap: float = 0.0,
                              slopes: torch.Tensor | None = None, causal: int = 0,
                              docs_q: torch.Tensor | None = None,
                              docs_k: torch.Tensor | None = None,
                              prefix: torch.Tensor | None = None,
                              lengths: torch.Tensor | None = None,
                              out: torch.Tensor | None = None,
                              status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """decay * weights + the attention weight every cached key received from q's rows (summed over
    the heads that share its key head): fp32 [B, Hk, Nk].  lse, scale and the masks as in the forward
    that wrote lse.  weights None starts from zero; out=weights accumulates in place; entries past
    lengths[b] stay as they were (zero when there were none)."""
    dev = q.get_device()
    if dev >= 0 and (stream is not None or dev != _current_device()):
        return _elsewhere(dev, stream, sparse_attn_cache_weights, q, k, lse, weights, decay=decay,
                          scale=scale, cap=cap, slopes=slopes, causal=causal, docs_q=docs_q,
                          docs_k=docs_k, prefix=prefix, lengths=lengths, out=out, status=status)
    qs, ks = _view(q, _bf16, "q", dev), _view(k, _bf16, "k", dev)
    n, sl, dq, dk, px, lens, made = _mask_fields(q, k, dev, slopes, docs_q, docs_k, prefix, lengths)
    B, H, Nq, d = q.shape
    shape = k.shape[:3]
    if out is None:
        make = torch.zeros if weights is None and lengths is not None else torch.empty
        out = make(shape, dtype=_f32, device=q.device)
    p = _MASKED.pack(B, H, shape[1], Nq, shape[2], d, 1.0 / math.sqrt(d) if scale is None else scale, 0,
                     *qs, *ks, 0, 0, 0, 0, 0, 0, cap, sl, causal, n, dq, dk, px, lens)
    st = _c_weights(p, q.data_ptr(), k.data_ptr(), _flat(lse, _f32, "lse", dev, (B, H, Nq)),
                    _flat(weights, _f32, "weights", dev, shape),
                    _flat(out, _f32, "out", dev, shape), 0.0 if weights is None else decay,
                    0 if status is None else _flat(status, _i32, "status", dev),
                    _current_stream(dev))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_cache_weights")
    return out


def sparse_attn_cache_evict(weights: torch.Tensor, k: torch.Tensor | None, v: torch.Tensor | None,
                            budget: int, *, sink: int = 0, recent: int = 0,
                            lengths: torch.Tensor | None = None, out=None,
                            kept: torch.Tensor | None = None, stream=None):
    """Keeps min(n, budget) of every head's n = lengths[b] (default: all) cached entries: the first
    `sink`, the last `recent` and the largest weights between (ties: the lowest index).

    weights fp32 [B, Hk, Nk]; k, v bf16 views [B, Hk, Nk, d], or None to select only.  Returns (kept
    int32 [B, Hk, budget], k, v [B, Hk, budget, d], weights [B, Hk, budget]): the kept entries in their
    order; behind a shorter one kept is -1 and the rows of `out` = (k, v, weights) are left as they
    were (zero when out is not given)."""
    dev = weights.get_device()
    if dev >= 0 and (stream is not None or dev != _current_device()):
        return _elsewhere(dev, stream, sparse_attn_cache_evict, weights, k, v, budget, sink=sink,
                          recent=recent, lengths=lengths, out=out, kept=kept)
    if weights.dim() != 3 or dev < 0:
        raise ValueError("weights must be a CUDA tensor [B, Hk, Nk]")
    B, H, N = weights.shape
    if (k is None) != (v is None):
        raise ValueError("k and v come together")
    if budget < 1:
        raise ValueError("budget must be at least 1")
    w = _flat(weights, _f32, "weights", dev)
    lens = _flat(lengths, _i32, "lengths", dev, (B,))
    d = 128
    strides = (0,) * 12
    if k is not None:
        ks, vs = _view(k, _bf16, "k", dev), _view(v, _bf16, "v", dev)
        d = k.shape[3]
        if k.shape != v.shape or k.shape[:3] != weights.shape:
            raise ValueError("k and v must be [B, Hk, Nk, d] with weights' B, Hk and Nk")
    if out is None:
        make = torch.empty if lengths is None and budget <= N else torch.zeros
        ko = vo = None
        if k is not None:
            ko, vo = (make((B, H, budget, d), dtype=_bf16, device=weights.device) for _ in range(2))
        wo = make((B, H, budget), dtype=_f32, device=weights.device)
    else:
        ko, vo, wo = out
    if kept is None:
        kept = torch.empty((B, H, budget), dtype=_i32, device=weights.device)
    kp = vp = kop = vop = 0
    if k is not None:
        if ko.shape != (B, H, budget, d) or vo.shape != ko.shape:
            raise ValueError("out must hold k and v as [B, Hk, budget, d]")
        strides = (*ks, *vs, *_view(ko, _bf16, "out", dev), *_view(vo, _bf16, "out", dev))
        kp, vp, kop, vop = k.data_ptr(), v.data_ptr(), ko.data_ptr(), vo.data_ptr()
    st = _c_evict(_EVICT.pack(B, H, N, d, budget, sink, recent, lens, *strides), w, kp, vp,
                  _flat(kept, _i32, "kept", dev, (B, H, budget)), kop, vop,
                  _flat(wo, _f32, "out", dev, (B, H, budget)),
                  _current_stream(dev))
    if st != SA_OK:
        raise SparseAttnError(st, "sparse_attn_cache_evict")
    return kept, ko, vo, wo


class HostLayer:
    """One attention layer from pinned host tensors (sparse_attn_layer_from_host):
    device staging, one chunk's scratch and two copy streams, allocated once
    for a shape.  Calling it enqueues the copies in, the build + forward per
    chunk of heads and the copies out; `synchronize()` waits for the layer."""

    def __init__(self, B, H, Nq, Nk, d, *, group_size=128, mode="topk", topk=0, threshold=0.0,
                 mass=0.99, heads_per_chunk=0, out_dtype=torch.bfloat16, with_lse=True,
                 device=None):
        dev = torch.device(device or "cuda")
        self.p = sa_problem(B, H, Nq, Nk, d, group_size, 1.0 / math.sqrt(d), _OUT[out_dtype])
        m = _MODES.get(mode, mode)
        self.sel = sa_select(m, int(topk), float(threshold), float(mass))
        BH = B * H
        mid = BH - 2 if BH > 2 else 0
        self.hc = heads_per_chunk if heads_per_chunk > 0 else (-(-mid // 3) if mid > 0 else BH)
        self.hc = min(self.hc, BH)
        G = -(-Nq // group_size)
        kmax = min(max(int(topk), 1), Nk) if m == SA_SELECT_TOPK else Nk
        cp = sa_problem(1, self.hc, Nq, Nk, d, group_size, self.p.scale, self.p.out_dtype)
        self.ws = torch.empty(sparse_attn_build_index_workspace_size(cp), dtype=torch.uint8, device=dev)
        self.row_ptr = torch.empty(self.hc * G + 1, dtype=torch.int64, device=dev)
        self.cap = self.hc * G * kmax
        self.col = torch.empty(self.cap, dtype=torch.int32, device=dev)
        self.q = torch.empty(B, H, Nq, d, dtype=torch.bfloat16, device=dev)
        self.k = torch.empty(B, H, Nk, d, dtype=torch.bfloat16, device=dev)
        self.v = torch.empty_like(self.k)
        self.o = torch.empty(B, H, Nq, d, dtype=out_dtype, device=dev)
        self.lse = torch.empty(B, H, Nq, dtype=torch.float32, device=dev) if with_lse else None
        self.copy_in = torch.cuda.Stream(device=dev)
        self.copy_out = torch.cuda.Stream(device=dev)

    def __call__(self, q_host, k_host, v_host, o_host, lse_host=None, stream=None):
        for t in (q_host, k_host, v_host, o_host):
            if t.is_cuda or not t.is_contiguous():
                raise ValueError("host tensors must be contiguous CPU tensors (pinned to overlap)")
        if (lse_host is None) != (self.lse is None):
            raise ValueError("lse_host must be given exactly when the layer keeps lse")
        st = lib.sparse_attn_layer_from_host(
            ctypes.byref(self.p), ctypes.byref(self.sel), _ptr(q_host), _ptr(k_host), _ptr(v_host),
            _ptr(o_host), _ptr(lse_host), _ptr(self.q), _ptr(self.k), _ptr(self.v), _ptr(self.o),
            _ptr(self.lse), _ptr(self.row_ptr), _ptr(self.col), self.cap, _ptr(self.ws),
            self.ws.numel(), int(self.hc), _stream(stream), _stream(self.copy_in),
            _stream(self.copy_out))
        if st != SA_OK:
            raise SparseAttnError(st, "sparse_attn_layer_from_host")

    def synchronize(self, stream=None):
        (stream if stream is not None else torch.cuda.current_stream()).synchronize()


# Short aliases for Python callers.
build_index = sparse_attn_build_index
build_index_dense = sparse_attn_build_index_dense
forward = sparse_attn_forward
forward_delta = sparse_attn_forward_delta
validate_index = sparse_attn_validate_index
voxel_permute = sparse_attn_voxel_permute
index_from_bitmask = sparse_attn_index_from_bitmask
index_from_block_mask = sparse_attn_index_from_block_mask
kv_window_append = sparse_attn_kv_window_append
rope = sparse_attn_rope
forward_masked = sparse_attn_forward_masked
cache_weights = sparse_attn_cache_weights
cache_evict = sparse_attn_cache_evict
