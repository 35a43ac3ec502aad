"""Routed block-sparse self-attention on GB300 (sm_103a): Python binding.

This module only marshals arguments to the C ABI of ``libsa_gb300.so``
(declared in ``include/sa.h``): it reads tensor pointers, strides and the
current CUDA stream, allocates outputs with torch when the caller passes
none, and calls the library. Every step of routing and attention runs in the
library's CUDA kernels. There is no CPU path: if the library is missing or a
tensor is not on a CUDA device, the call raises.

Entry points (same names as the C ABI):
    sa_route(q, k, prefix_len, tau, ...)              -> (row_ptr, col_idx)
    sa_attn_sparse(q, k, v, row_ptr, col_idx, ...)    -> (o, lse)
    sa_attn_dense(q, k, v, ...)                       -> (o, lse)
    sa_qk_prologue(q, k, ...)                         -> (q_out, k_out, workspace)
    sa_qk_quantize(q, k, ...)                         -> (q8, k8, q_exp, k_exp)
    sa_route_pooled(q_out, workspace, prefix_len, tau, ...) -> (row_ptr, col_idx)
    sa_forward_host(q_host, k_host, v_host, ...)      -> o_host (+ lse_host)
Over a paged key-value cache (one new token per sequence and call):
    sa_cache_append(k, v, k_cache, v_cache, page_table, seq_lens, ...) -> q_out
    sa_route_pages(q, k_sum, page_table, seq_lens, prefix_len, budget) -> (row_ptr, col_idx)
    sa_attn_decode(q, k_cache, v_cache, page_table, seq_lens, ...)     -> (o, lse)
A few drafted tokens per sequence and call:
    sa_attn_tree(q, k_cache, v_cache, page_table, seq_lens, parents=...) -> (o, lse)
    sa_cache_accept(k_cache, v_cache, page_table, seq_lens, path, path_lens, ...)
The pool's pages:
    sa_pages_fork(page_table, seq_lens, refs, src, ...)  -> the forked table, lengths, refs, moves
    sa_pages_resize(page_table, refs, seq_lens, more)
    sa_pages_compact(page_table, refs, ...)              -> table, refs, moves, pages in use
    sa_cache_copy(k_cache, v_cache, moves, n_moves, ...)
Tensors are [B, S, H, D] bf16 with a contiguous last dimension.
"""

from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from typing import Optional, Tuple

import torch

__all__ = [
    "SaError", "load_library", "library_path", "sa_params", "make_params", "sa_route",
    "sa_qk_prologue", "sa_route_pooled", "sa_attn_prepare", "sa_attn_run",
    "sa_attn_sparse", "sa_attn_dense", "sa_forward_host", "sa_route_workspace_bytes",
    "sa_attn_workspace_bytes", "sa_route_max_nnz", "check_dev_status", "EXPORTS",
    "sa_qk_quantize", "SA_QK_BF16", "SA_QK_FP8", "QK_FORMATS",
    "SA_DEV_CAPACITY", "SA_DEV_TIMEOUT", "SA_DEV_BAD_ROUTE", "SA_DEV_RANGE",
    "SA_ROUTE_THRESHOLD", "SA_ROUTE_DENSE_PREFIX_QUERIES", "SA_ROUTE_TOP_MASS", "ROUTE_MODES",
    "sa_cache_params", "make_cache_params", "sa_cache_append", "sa_route_pages", "sa_attn_decode",
    "sa_route_pages_max_nnz", "sa_route_pages_workspace_bytes", "sa_attn_decode_workspace_bytes",
    "SA_DEV_BAD_CACHE", "SA_CACHE_BF16", "SA_CACHE_FP8", "CACHE_FORMATS", "SA_ROPE_INTERLEAVED",
    "SA_ROPE_HALF", "ROPE_LAYOUTS", "sa_rope_axes", "sa_attn_tree", "sa_attn_tree_workspace_bytes",
    "sa_cache_accept", "sa_cache_copy", "sa_pages_fork", "sa_pages_resize", "sa_pages_compact",
    "sa_pages_workspace_bytes", "SA_DEV_BAD_TREE", "SA_ROPE_STAYS", "SA_TREE_MAX",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB = None

SA_OK, SA_ERR_INVALID_ARG, SA_ERR_UNSUPPORTED, SA_ERR_CAPACITY, SA_ERR_CUDA, SA_ERR_TIMEOUT = range(6)
SA_DEV_CAPACITY, SA_DEV_TIMEOUT, SA_DEV_BAD_ROUTE, SA_DEV_RANGE = 1, 2, 4, 8
SA_DEV_BAD_CACHE, SA_DEV_BAD_TREE = 16, 32
# readings of the router rule (sa_params.route_mode)
SA_ROUTE_THRESHOLD, SA_ROUTE_DENSE_PREFIX_QUERIES, SA_ROUTE_TOP_MASS = 0, 1, 2
ROUTE_MODES = {"threshold": SA_ROUTE_THRESHOLD,
               "dense_prefix_queries": SA_ROUTE_DENSE_PREFIX_QUERIES,
               "top_mass": SA_ROUTE_TOP_MASS}
# arithmetic of the score product (sa_params.qk_format)
SA_QK_BF16, SA_QK_FP8 = 0, 1
QK_FORMATS = {"bf16": SA_QK_BF16, "fp8": SA_QK_FP8}
# storage of a paged cache (sa_cache_params.cache_format), by the tensors' dtype
SA_CACHE_BF16, SA_CACHE_FP8 = 0, 1
CACHE_FORMATS = {torch.bfloat16: SA_CACHE_BF16, torch.float8_e4m3fn: SA_CACHE_FP8,
                 torch.uint8: SA_CACHE_FP8}
# which elements of a head vector the rotation pairs (sa_cache_params.rope_layout)
SA_ROPE_INTERLEAVED, SA_ROPE_HALF = 0, 1
ROPE_LAYOUTS = {"interleaved": SA_ROPE_INTERLEAVED, "half": SA_ROPE_HALF}
SA_ROPE_STAYS = 255        # a pair that no axis turns
PAGE = 64
SA_TREE_MAX = 64           # most new tokens of a sequence in sa_attn_tree

# Every function include/sa.h declares.
EXPORTS = (
    "sa_params_init", "sa_num_blocks", "sa_route_rows", "sa_route_max_nnz",
    "sa_route_workspace_bytes", "sa_route", "sa_attn_workspace_bytes", "sa_attn_sparse",
    "sa_attn_dense", "sa_forward_host", "sa_dev_status_decode", "sa_status_string",
    "sa_route_static", "sa_qk_prologue", "sa_route_pooled", "sa_check_wait_timeout",
    "sa_attn_prepare", "sa_attn_run", "sa_qk_quantize",
    "sa_cache_params_init", "sa_cache_append", "sa_route_pages", "sa_route_pages_max_nnz",
    "sa_route_pages_workspace_bytes", "sa_attn_decode", "sa_attn_decode_workspace_bytes",
    "sa_qk_prologue_axes", "sa_cache_append_axes", "sa_attn_tree", "sa_attn_tree_workspace_bytes",
    "sa_cache_accept", "sa_cache_copy", "sa_pages_workspace_bytes", "sa_pages_fork",
    "sa_pages_resize", "sa_pages_compact",
)
SA_ROUTE_STATIC_WS_BYTES = 32 << 20


class SaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_status_name(code)}")


class sa_params(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("S", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
        ("block", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
        ("tau", ctypes.c_float), ("softmax_scale", ctypes.c_float),
        ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3), ("o_stride", ctypes.c_int64 * 3),
        ("route_mode", ctypes.c_int32), ("q_block", ctypes.c_int32),
        ("qk_format", ctypes.c_int32),
    ]


class sa_cache_params(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in (
        "B", "S", "H", "H_kv", "D", "page", "n_pages", "max_pages", "cache_format", "prefix_len",
        "page_budget", "qk_norm", "rope_layout", "rope_rows")] + [
        ("eps", ctypes.c_float), ("softmax_scale", ctypes.c_float),
        ("table_stride", ctypes.c_int64)] + [(name, ctypes.c_int64 * 3) for name in (
            "q_stride", "k_stride", "v_stride", "o_stride", "kc_stride", "vc_stride")]


class sa_rope_axes(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("pos_stride", ctypes.c_int64 * 2),
                ("n_axes", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("axis_of", ctypes.c_uint8 * 64)]


def library_path() -> str:
    return os.path.join(_PKG, "libsa_gb300.so")


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load (once) and type the shared library. Raises if it is missing."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or library_path()
    if not os.path.exists(p):
        raise FileNotFoundError(
            f"{p} is missing: build it with `python -m block_sparse_attention_sa_gb300.build`")
    lib = ctypes.CDLL(p)
    P = ctypes.POINTER(sa_params)
    vp, i32p, i64, sz = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_int64, ctypes.c_size_t
    sig = {
        "sa_params_init": (None, [P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.c_int32, ctypes.c_float]),
        "sa_num_blocks": (ctypes.c_int32, [P]),
        "sa_route_rows": (i64, [P]),
        "sa_route_max_nnz": (i64, [P]),
        "sa_route_workspace_bytes": (sz, [P]),
        "sa_attn_workspace_bytes": (sz, [P]),
        "sa_route": (ctypes.c_int, [P, vp, vp, vp, vp, i64, vp, sz, vp, vp]),
        "sa_route_static": (ctypes.c_int, [P, vp, vp, vp, vp, i64, vp, vp]),
        "sa_qk_prologue": (ctypes.c_int, [P, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp,
                                          sz, vp, vp]),
        "sa_route_pooled": (ctypes.c_int, [P, vp, vp, i64, vp, sz, vp, vp]),
        "sa_attn_sparse": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "sa_attn_dense": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "sa_forward_host": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64,
                                           vp, sz, vp, vp]),
        "sa_dev_status_decode": (ctypes.c_int, [ctypes.c_int32]),
        "sa_check_wait_timeout": (ctypes.c_int, [vp, vp]),
        "sa_attn_prepare": (ctypes.c_int, [P, vp, vp, vp, vp, sz, vp, vp]),
        "sa_attn_run": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "sa_qk_quantize": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp]),
        "sa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    }
    C, i32 = ctypes.POINTER(sa_cache_params), ctypes.c_int32
    sig.update({
        "sa_cache_params_init": (None, [C] + [i32] * 6),
        "sa_cache_append": (ctypes.c_int, [C] + [vp] * 19),
        "sa_route_pages_max_nnz": (i64, [C]),
        "sa_route_pages_workspace_bytes": (sz, [C]),
        "sa_route_pages": (ctypes.c_int, [C] + [vp] * 6 + [i64, vp, sz, vp, vp]),
        "sa_attn_decode_workspace_bytes": (sz, [C]),
        "sa_attn_decode": (ctypes.c_int, [C] + [vp] * 9 + [i64, vp, vp, vp, sz, vp, vp]),
    })
    X, i32 = ctypes.POINTER(sa_rope_axes), ctypes.c_int32
    sig.update({
        "sa_qk_prologue_axes": (ctypes.c_int, [P, vp, vp, i32, vp, vp, ctypes.c_float, vp, vp, X,
                                               vp, vp, vp, sz, vp, vp]),
        "sa_cache_append_axes": (ctypes.c_int, [C] + [vp] * 8 + [X] + [vp] * 11),
        "sa_attn_tree_workspace_bytes": (sz, [C]),
        "sa_attn_tree": (ctypes.c_int, [C] + [vp] * 9 + [i64, vp, vp, i64, vp, vp, vp, sz, vp, vp]),
        "sa_cache_accept": (ctypes.c_int, [C] + [vp] * 7 + [i64] + [vp] * 4),
        "sa_cache_copy": (ctypes.c_int, [C] + [vp] * 4 + [i64, vp, vp, vp]),
        "sa_pages_workspace_bytes": (sz, [i32, i32]),
        "sa_pages_fork": (ctypes.c_int, [i32] * 4 + [vp, i64, vp, vp, vp, vp, i64, vp, vp, vp, vp,
                                                     vp, sz, vp, vp]),
        "sa_pages_resize": (ctypes.c_int, [i32] * 3 + [vp, i64, vp, vp, vp, i32, vp, sz, vp, vp]),
        "sa_pages_compact": (ctypes.c_int, [i32] * 3 + [vp, i64, vp, vp, i64, vp, vp, vp, vp, vp,
                                                        sz, vp, vp]),
    })
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _LIB = lib
    return lib


def _status_name(code: int) -> str:
    try:
        return load_library().sa_status_string(code).decode()
    except Exception:  # library not loadable: still report the number
        return f"status {code}"


def _check(code: int, what: str) -> None:
    if code != SA_OK:
        raise SaError(code, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _bshd_strides(t: torch.Tensor, name: str):
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be [B, S, H, D] with a contiguous last dimension")
    return (t.stride(0), t.stride(1), t.stride(2))


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device: there is no CPU path")


def make_params(q: torch.Tensor, k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                o: Optional[torch.Tensor] = None, prefix_len: int = 0, tau: float = 1.0,
                scale: float = 0.0, mode="threshold", q_block: int = 64,
                qk_format="bf16") -> sa_params:
    B, S, H, D = q.shape
    p = sa_params()
    p.B, p.S, p.H, p.D, p.block, p.q_block = B, S, H, D, 64, int(q_block)
    p.qk_format = QK_FORMATS[qk_format] if isinstance(qk_format, str) else int(qk_format)
    p.prefix_len, p.tau, p.softmax_scale = int(prefix_len), float(tau), float(scale)
    p.route_mode = ROUTE_MODES[mode] if isinstance(mode, str) else int(mode)
    for field, t in (("q_stride", q), ("k_stride", k if k is not None else q),
                     ("v_stride", v if v is not None else q), ("o_stride", o if o is not None else q)):
        st = _bshd_strides(t, field[0])
        arr = getattr(p, field)
        for i in range(3):
            arr[i] = st[i]
    return p


def sa_route_workspace_bytes(p: sa_params) -> int:
    return int(load_library().sa_route_workspace_bytes(ctypes.byref(p)))


def sa_attn_workspace_bytes(p: sa_params) -> int:
    return int(load_library().sa_attn_workspace_bytes(ctypes.byref(p)))


def sa_route_max_nnz(p: sa_params) -> int:
    return int(load_library().sa_route_max_nnz(ctypes.byref(p)))


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError("workspace too small")
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def sa_route(q: torch.Tensor, k: torch.Tensor, prefix_len: int, tau: float, scale: float = 0.0, *,
             mode="threshold", q_block: int = 64, row_ptr: Optional[torch.Tensor] = None,
             col_idx: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             dev_status: Optional[torch.Tensor] = None,
             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Block route of every (b, h, query block): int32 row_ptr [B*H*Nb+1] and
    col_idx (capacity B*H*Nb*Nb unless given; valid entries are
    col_idx[:row_ptr[-1]]). ``mode``: "threshold", "dense_prefix_queries" or
    "top_mass" (the SA_ROUTE_* readings of sa.h). ``q_block``: 64, or 128 for
    128-token query blocks (rows 2i and 2i + 1 then hold the same list)."""
    _require_cuda(q, k)
    lib = load_library()
    p = make_params(q, k, prefix_len=prefix_len, tau=tau, scale=scale, mode=mode,
                    q_block=q_block)
    rows = int(lib.sa_route_rows(ctypes.byref(p)))
    if rows == 0:
        _check(SA_ERR_INVALID_ARG, "sa_route")
    if row_ptr is None:
        row_ptr = torch.empty(rows + 1, dtype=torch.int32, device=q.device)
    if col_idx is None:
        col_idx = torch.empty(sa_route_max_nnz(p), dtype=torch.int32, device=q.device)
    ws = _workspace(sa_route_workspace_bytes(p), q.device, workspace)
    code = lib.sa_route(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(row_ptr), _ptr(col_idx),
                        col_idx.numel(), _ptr(ws), ws.numel() * ws.element_size(),
                        _ptr(dev_status), _stream(stream))
    _check(code, "sa_route")
    return row_ptr, col_idx


@functools.lru_cache(maxsize=64)
def _axis_bytes(axes: tuple, n_axes: Optional[int], D: int):
    """The axis of each of the D/2 pairs as bytes, and how many axes there are."""
    if len(axes) == D // 2 and n_axes != D // 2:
        of, n = list(axes), max(axes) + 1 if n_axes is None else n_axes
        if any(a < -1 or a >= n for a in of):
            raise ValueError(f"axes of the pairs must be -1 or one of {n}")
        of = [SA_ROPE_STAYS if a < 0 else a for a in of]
    else:
        n = len(axes)
        if any(a < 0 for a in axes) or sum(axes) > D // 2 or (n_axes is not None and n_axes != n):
            raise ValueError("axes must give the pairs of each axis of positions, at most D/2 "
                             "in all, or the axis of each of the D/2 pairs")
        of = [a for a, k in enumerate(axes) for _ in range(k)]
        of += [SA_ROPE_STAYS] * (D // 2 - len(of))
    if not 1 <= n <= 8:
        raise ValueError("positions have 1 to 8 axes")
    return bytes(of), n


def _axes_of(axes, positions: Optional[torch.Tensor], D: int):
    """((bytes, number of axes), positions [B, S, n_axes] or None) of what a caller gives."""
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dim() not in (2, 3):
            raise ValueError("positions must be int32 [B, S, n_axes], or [B, S] for one axis")
        if positions.dim() == 2:
            positions = positions[..., None]
    n = None if positions is None else positions.shape[2]
    if axes is None:
        if n not in (None, 1):
            raise ValueError("positions with several axes go with axes")
        axes = (D // 2,)
    return _axis_bytes(tuple(int(a) for a in axes), n, D), positions


def _rope_axes(of, positions: Optional[torch.Tensor], cos, sin, q: torch.Tensor) -> sa_rope_axes:
    B, S, _, D = q.shape
    if (cos is None or sin is None or cos.dim() != 2 or cos.shape[0] < 1
            or cos.shape[1] != D // 2 or sin.shape != cos.shape):
        raise ValueError("cos and sin must be fp32 [rows, D/2] with rows >= 1")
    x = sa_rope_axes()
    x.axis_of[: D // 2] = of[0]
    x.n_axes, x.rows = of[1], cos.shape[0]
    if positions is not None:
        if (positions.dtype != torch.int32 or positions.shape != (B, S, of[1])
                or (positions.stride(2) != 1 and of[1] != 1)):
            raise ValueError(f"positions must be int32 [{B}, {S}, {of[1]}], the axes contiguous")
        x.positions = positions.data_ptr()
        x.pos_stride[:] = positions.stride()[:2]
    return x


def sa_qk_prologue(q: torch.Tensor, k: torch.Tensor, gamma_q: Optional[torch.Tensor] = None,
                   gamma_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
                   qk_norm: bool = True, positions: Optional[torch.Tensor] = None, axes=None,
                   q_block: int = 64, q_out: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    """QK-norm + RoPE of q, k (bf16 [B,S,H,D]) with the router's pooling fused
    in: returns (q_out, k_out, workspace); pass the workspace to
    sa_route_pooled. gamma_* fp32 [D] or None; cos, sin fp32 [S, D/2] or None.
    q_out/k_out default to new tensors with q/k's strides; pass q_out=q for in place.
    Positions with several axes (time, height, width): ``positions`` int32 [B, S, n_axes]
    (or [B, S] for one axis) pick each pair's row of cos, sin fp32 [rows, D/2]; ``axes``
    gives the number of pairs of each axis, first axis first (pairs behind the last are
    not turned), or the axis of each of the D/2 pairs (-1: not turned). Without
    ``positions`` a token's place counts on every axis. ``qk_norm`` = False leaves the
    norm out."""
    _require_cuda(q, k, gamma_q, gamma_k, cos, sin, positions)
    by_axes = positions is not None or axes is not None or not qk_norm
    if by_axes:
        of, pos = _axes_of(axes, positions, q.shape[-1])
    lib = load_library()
    if q_out is None:
        q_out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=k.device)
    if q_out.stride() != q.stride() or k_out.stride() != k.stride():
        raise ValueError("q_out / k_out must have the strides of q / k")
    for t, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k"), (cos, "cos"), (sin, "sin")):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous fp32 tensor")
    # the kernels read and write q's shape of each
    for t, name in ((q, "q"), (k, "k"), (q_out, "q_out"), (k_out, "k_out")):
        if (t.dtype != torch.bfloat16 or t.dim() != 4 or t.shape[3] != q.shape[3]
                or any(a < b for a, b in zip(t.shape, q.shape))):
            raise ValueError(f"{name} must be bf16 with q's shape [B, S, H, D]")
    for t, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        if t is not None and t.numel() < q.shape[3]:
            raise ValueError(f"{name} must have D elements")
    for t, name in ((cos, "cos"), (sin, "sin")):
        if t is not None and not by_axes and t.numel() < q.shape[1] * (q.shape[3] // 2):
            raise ValueError(f"{name} must be [S, D/2]")
    _require_cuda(q_out, k_out, workspace, dev_status)
    if dev_status is not None and (dev_status.dtype != torch.int32 or dev_status.numel() < 1):
        raise ValueError("dev_status must be an int32 tensor")
    p = make_params(q, k, q_block=q_block)
    ws = _workspace(sa_route_workspace_bytes(p), q.device, workspace)
    if by_axes:
        x = _rope_axes(of, pos, cos, sin, q)
        with torch.cuda.device(q.device):
            code = lib.sa_qk_prologue_axes(
                ctypes.byref(p), _ptr(q), _ptr(k), 1 if qk_norm else 0, _ptr(gamma_q),
                _ptr(gamma_k), float(eps), _ptr(cos), _ptr(sin), ctypes.byref(x), _ptr(q_out),
                _ptr(k_out), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
                _stream(stream))
        _check(code, "sa_qk_prologue")
        return q_out, k_out, ws
    code = lib.sa_qk_prologue(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(gamma_q), _ptr(gamma_k),
                              float(eps), _ptr(cos), _ptr(sin), _ptr(q_out), _ptr(k_out), _ptr(ws),
                              ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream))
    _check(code, "sa_qk_prologue")
    return q_out, k_out, ws


def sa_route_pooled(q: torch.Tensor, workspace: torch.Tensor, prefix_len: int, tau: float,
                    scale: float = 0.0, *, k: Optional[torch.Tensor] = None, mode="threshold",
                    q_block: int = 64, row_ptr: Optional[torch.Tensor] = None,
                    col_idx: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None):
    """The route from the block means sa_qk_prologue left in ``workspace``;
    q (and k, default q's layout) give the shape and strides of that call."""
    _require_cuda(q, workspace)
    lib = load_library()
    p = make_params(q, k if k is not None else q, prefix_len=prefix_len, tau=tau, scale=scale,
                    mode=mode, q_block=q_block)
    rows = int(lib.sa_route_rows(ctypes.byref(p)))
    if rows == 0:
        _check(SA_ERR_INVALID_ARG, "sa_route_pooled")
    if row_ptr is None:
        row_ptr = torch.empty(rows + 1, dtype=torch.int32, device=q.device)
    if col_idx is None:
        col_idx = torch.empty(sa_route_max_nnz(p), dtype=torch.int32, device=q.device)
    code = lib.sa_route_pooled(ctypes.byref(p), _ptr(row_ptr), _ptr(col_idx), col_idx.numel(),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _ptr(dev_status), _stream(stream))
    _check(code, "sa_route_pooled")
    return row_ptr, col_idx


def _attn_out(q, o, lse, want_lse):
    B, S, H, D = q.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    return o, lse


def sa_attn_sparse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, row_ptr: torch.Tensor,
                   col_idx: torch.Tensor, scale: float = 0.0, *, o: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                   workspace: Optional[torch.Tensor] = None, q_block: int = 64,
                   qk_format="bf16", dev_status: Optional[torch.Tensor] = None, stream=None):
    """Attention over the routed key blocks: (o bf16 [B,S,H,D], lse fp32 [B,H,S] or None).
    ``q_block`` = 128 when the route came from sa_route(..., q_block=128): the
    kernel's tiles are then the 128-token query blocks, with no pairing step.
    ``qk_format`` = "fp8" for 8-bit scores (see sa_qk_quantize)."""
    _require_cuda(q, k, v, row_ptr, col_idx)
    lib = load_library()
    o, lse = _attn_out(q, o, lse, want_lse)
    p = make_params(q, k, v, o, scale=scale, q_block=q_block, qk_format=qk_format)
    ws = _workspace(sa_attn_workspace_bytes(p), q.device, workspace)
    code = lib.sa_attn_sparse(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr),
                              _ptr(col_idx), _ptr(o), _ptr(lse), _ptr(ws),
                              ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream))
    _check(code, "sa_attn_sparse")
    return o, lse


def sa_attn_prepare(v: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor, *,
                    workspace: torch.Tensor, q_block: int = 64, qk_format="bf16",
                    dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """First half of sa_attn_sparse: V repacked into ``workspace`` and the
    tile pairs chosen from the route. Returns the workspace."""
    _require_cuda(v, row_ptr, col_idx, workspace)
    p = make_params(v, v, v, v, q_block=q_block, qk_format=qk_format)
    if workspace.numel() * workspace.element_size() < sa_attn_workspace_bytes(p):
        raise ValueError("workspace too small")
    code = load_library().sa_attn_prepare(ctypes.byref(p), _ptr(v), _ptr(row_ptr), _ptr(col_idx),
                                          _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _ptr(dev_status), _stream(stream))
    _check(code, "sa_attn_prepare")
    return workspace


def sa_attn_run(q: torch.Tensor, k: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                scale: float = 0.0, *, workspace: torch.Tensor, v_like: Optional[torch.Tensor] = None,
                o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                want_lse: bool = True, q_block: int = 64, qk_format="bf16",
                dev_status: Optional[torch.Tensor] = None, stream=None):
    """Second half of sa_attn_sparse: the attention kernel over a workspace
    sa_attn_prepare filled (with 8-bit scores, after quantising q and k into
    it). ``v_like`` gives V's strides (default q's)."""
    _require_cuda(q, k, row_ptr, col_idx, workspace)
    o, lse = _attn_out(q, o, lse, want_lse)
    p = make_params(q, k, v_like, o, scale=scale, q_block=q_block, qk_format=qk_format)
    code = load_library().sa_attn_run(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(row_ptr),
                                      _ptr(col_idx), _ptr(o), _ptr(lse), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(),
                                      _ptr(dev_status), _stream(stream))
    _check(code, "sa_attn_run")
    return o, lse


def sa_qk_quantize(q: torch.Tensor, k: torch.Tensor, *,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    """The e4m3 codes of q and k (uint8 [B,S,H,D]) and the scale exponents of
    their 64-token blocks (int8 [B,H,Nb]); see sa.h."""
    _require_cuda(q, k)
    B, S, H, D = q.shape
    nb = (S + 63) // 64
    q8 = torch.empty((B, S, H, D), dtype=torch.uint8, device=q.device)
    k8 = torch.empty_like(q8)
    qe = torch.empty((B, H, nb), dtype=torch.int8, device=q.device)
    ke = torch.empty_like(qe)
    p = make_params(q, k)
    code = load_library().sa_qk_quantize(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(q8), _ptr(k8),
                                         _ptr(qe), _ptr(ke), _ptr(dev_status), _stream(stream))
    _check(code, "sa_qk_quantize")
    return q8, k8, qe, ke


def sa_attn_dense(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float = 0.0, *,
                  o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  want_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                  qk_format="bf16", dev_status: Optional[torch.Tensor] = None, stream=None):
    """Attention over every key block (density 100%)."""
    _require_cuda(q, k, v)
    lib = load_library()
    o, lse = _attn_out(q, o, lse, want_lse)
    p = make_params(q, k, v, o, scale=scale, qk_format=qk_format)
    ws = _workspace(sa_attn_workspace_bytes(p), q.device, workspace)
    code = lib.sa_attn_dense(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                             _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
                             _stream(stream))
    _check(code, "sa_attn_dense")
    return o, lse


def sa_forward_host(q_host: torch.Tensor, k_host: torch.Tensor, v_host: torch.Tensor,
                    prefix_len: int, tau: float, scale: float = 0.0, *, bufs: dict,
                    mode="threshold", q_block: int = 64, o_host: Optional[torch.Tensor] = None,
                    lse_host: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One layer from (pinned) host tensors through the device buffers in
    ``bufs`` (q, k, v, o, lse, row_ptr, col_idx, ws, status); returns o_host.
    Enqueues only; synchronise the stream before reading o_host."""
    lib = load_library()
    if o_host is None:
        o_host = torch.empty_like(q_host, pin_memory=True)
    p = make_params(bufs["q"], prefix_len=prefix_len, tau=tau, scale=scale, mode=mode,
                    q_block=q_block)
    ws = bufs["ws"]
    code = lib.sa_forward_host(
        ctypes.byref(p), _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(o_host), _ptr(lse_host),
        _ptr(bufs["q"]), _ptr(bufs["k"]), _ptr(bufs["v"]), _ptr(bufs["o"]), _ptr(bufs.get("lse")),
        _ptr(bufs["row_ptr"]), _ptr(bufs["col_idx"]), bufs["col_idx"].numel(), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(bufs.get("status")), _stream(stream))
    _check(code, "sa_forward_host")
    return o_host


def alloc_layer_buffers(B: int, S: int, H: int, D: int, device="cuda", qk_format="bf16") -> dict:
    """Device buffers for sa_forward_host (one workspace sized for both calls)."""
    q = torch.empty((B, S, H, D), dtype=torch.bfloat16, device=device)
    p = make_params(q, qk_format=qk_format)
    bufs = {"q": q, "k": torch.empty_like(q), "v": torch.empty_like(q), "o": torch.empty_like(q),
            "lse": torch.empty((B, H, S), dtype=torch.float32, device=device),
            "row_ptr": torch.empty(int(load_library().sa_route_rows(ctypes.byref(p))) + 1,
                                   dtype=torch.int32, device=device),
            "col_idx": torch.empty(sa_route_max_nnz(p), dtype=torch.int32, device=device),
            "status": torch.zeros(1, dtype=torch.int32, device=device)}
    nbytes = max(sa_route_workspace_bytes(p), sa_attn_workspace_bytes(p))
    bufs["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return bufs


# ------------------------------------------------------ paged key-value cache --
#
# One call of these serves one token, so its own cost counts: tensors are checked
# and marshalled by the compiled module _sa_bind, which calls the same C ABI.

_BIND = None


def _bind():
    """The compiled module, attached to the library. Raises if it is missing."""
    global _BIND
    if _BIND is None:
        from . import build as _build

        path = _build.module_path()
        if not os.path.exists(path):
            raise FileNotFoundError(
                f"{path} is missing (one is built for each torch and Python): build it with "
                "`python -m block_sparse_attention_sa_gb300.build`")
        spec = importlib.util.spec_from_file_location("_sa_bind", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        lib = load_library()
        module.attach(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in
                        ("sa_cache_append", "sa_route_pages", "sa_attn_decode",
                         "sa_cache_append_axes", "sa_attn_tree", "sa_cache_accept",
                         "sa_cache_copy", "sa_pages_fork", "sa_pages_resize",
                         "sa_pages_compact")))
        _BIND = module
    return _BIND


def _call(what: str, fn, index: int, stream, *args) -> None:
    """fn(device, *args, raw stream) with the device of the tensors current."""
    raw = (torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))
    if index == torch._C._cuda_getDevice():
        code = fn(index, *args, raw)
    else:
        with torch.cuda.device(index):
            code = fn(index, *args, raw)
    if code:
        _check(code, what)


def _cuda_index(t: torch.Tensor) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device: there is no CPU path")
    return t.get_device()


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def make_cache_params(page_table: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                      k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                      o: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                      v_cache: Optional[torch.Tensor] = None,
                      k_sum: Optional[torch.Tensor] = None, scale: float = 0.0,
                      prefix_len: int = 0, budget: int = 0) -> sa_cache_params:
    """The parameters of a paged-cache call on these tensors (those it takes):
    q, k, v, o [B, S, heads, D]; k_cache, v_cache [n_pages, H_kv, 64, D] in
    bf16, or e4m3 as float8_e4m3fn or uint8; k_sum [n_pages, H_kv, D]."""
    p = sa_cache_params()
    pool = k_cache if k_cache is not None else k_sum
    if pool is None or pool.dim() != (4 if k_cache is not None else 3):
        raise ValueError("k_cache must be [n_pages, H_kv, 64, D], k_sum [n_pages, H_kv, D]")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    p.n_pages, p.H_kv, p.D = pool.shape[0], pool.shape[1], pool.shape[-1]
    p.B, p.max_pages = page_table.shape
    p.page, p.table_stride, p.eps = PAGE, page_table.stride(0), 1e-6
    p.prefix_len, p.page_budget, p.softmax_scale = int(prefix_len), int(budget), float(scale)
    for field, t in (("q_stride", q), ("k_stride", k), ("v_stride", v), ("o_stride", o)):
        if t is not None:
            getattr(p, field)[:] = _bshd_strides(t, field[0])
    tokens = q if q is not None else k
    p.S = 1 if tokens is None else tokens.shape[1]
    p.H = p.H_kv if q is None else q.shape[2]
    if k_cache is not None:
        if (v_cache is None or v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype
                or k_cache.shape[2] != PAGE or k_cache.stride(3) != 1 or v_cache.stride(3) != 1):
            raise ValueError("k_cache, v_cache must be alike, [n_pages, H_kv, 64, D] with a "
                             "contiguous last dimension")
        if k_cache.dtype not in CACHE_FORMATS:
            raise ValueError("k_cache, v_cache must be bfloat16, float8_e4m3fn or uint8 (e4m3)")
        p.cache_format = CACHE_FORMATS[k_cache.dtype]
        p.kc_stride[:], p.vc_stride[:] = k_cache.stride()[:3], v_cache.stride()[:3]
    return p


def sa_cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, *,
                    q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                    new_lens: Optional[torch.Tensor] = None, qk_norm: bool = False,
                    gamma_q: Optional[torch.Tensor] = None,
                    gamma_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
                    rope="interleaved", positions: Optional[torch.Tensor] = None, axes=None,
                    k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, k_sum: Optional[torch.Tensor] = None,
                    lens_out: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None,
                    stream=None) -> Optional[torch.Tensor]:
    """The new tokens' keys and values (bf16 [B, S, H_kv, D]) into the paged
    cache behind each sequence's ``seq_lens`` tokens, normed (``qk_norm``) and
    rotated (``cos``, ``sin`` fp32 [rows, D/2] by position; ``rope``
    "interleaved" or "half") on the way; see sa.h. With ``q`` [B, S, H, D]
    returns the queries normed and rotated alike (``q_out``, default new; pass
    q_out=q for in place). ``new_lens``: how many of the S tokens each sequence
    brings. ``k_sum`` gathers the per-page key sums that sa_route_pages reads (taking
    tokens back: keep a copy of the last page's, see sa.h); ``lens_out`` receives the
    new lengths. Rows of ``q_out`` of tokens that are not stored are not written.
    ``positions``, ``axes``: as in sa_qk_prologue; a token is rotated by its positions
    and stored behind its sequence all the same (drafted tokens: their depth; images:
    time, height, width)."""
    index = _cuda_index(k)
    of = (None, 0)
    if positions is not None or axes is not None:
        of, positions = _axes_of(axes, positions, k.shape[-1])
    if q is not None and q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    _call("sa_cache_append", _bind().append, index, stream, k, v, k_cache, v_cache, page_table,
          seq_lens, q, q_out, new_lens, 1 if qk_norm else 0, gamma_q, gamma_k, eps, cos, sin,
          ROPE_LAYOUTS[rope] if isinstance(rope, str) else rope, positions, of[0], of[1], k_scale,
          v_scale, k_sum, lens_out, dev_status)
    return q_out


def sa_route_pages_max_nnz(p: sa_cache_params) -> int:
    return int(load_library().sa_route_pages_max_nnz(ctypes.byref(p)))


def sa_route_pages_workspace_bytes(p: sa_cache_params) -> int:
    return int(load_library().sa_route_pages_workspace_bytes(ctypes.byref(p)))


def sa_attn_decode_workspace_bytes(p: sa_cache_params) -> int:
    return int(load_library().sa_attn_decode_workspace_bytes(ctypes.byref(p)))


def sa_route_pages(q: torch.Tensor, k_sum: torch.Tensor, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, prefix_len: int, budget: int, *,
                   row_ptr: Optional[torch.Tensor] = None,
                   col_idx: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   dev_status: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The pages one new token of each sequence attends (q bf16 [B, 1, H, D],
    k_sum from sa_cache_append): int32 row_ptr [B*H_kv+1] and col_idx (valid
    entries are col_idx[:row_ptr[-1]]), for sa_attn_decode. Kept per key-value
    head: the prefix's pages, the newest one, and the best-scoring others until
    ``budget`` are."""
    index = _cuda_index(q)
    if row_ptr is None or col_idx is None or workspace is None:
        p = make_cache_params(page_table, q=q, k_sum=k_sum, prefix_len=prefix_len, budget=budget)
        if row_ptr is None:
            row_ptr = _empty((p.B * p.H_kv + 1,), torch.int32, q.device, stream)
        if col_idx is None:
            col_idx = _empty((sa_route_pages_max_nnz(p),), torch.int32, q.device, stream)
        if workspace is None:
            workspace = _empty((max(256, sa_route_pages_workspace_bytes(p)),), torch.uint8,
                               q.device, stream)
    _call("sa_route_pages", _bind().route, index, stream, q, k_sum, page_table, seq_lens,
          prefix_len, budget, row_ptr, col_idx, workspace, dev_status)
    return row_ptr, col_idx


def sa_attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, scale: float = 0.0, *,
                   row_ptr: Optional[torch.Tensor] = None,
                   col_idx: Optional[torch.Tensor] = None,
                   k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                   workspace: Optional[torch.Tensor] = None,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    """Attention of one new token per sequence (q bf16 [B, 1, H, D]) over its
    ``seq_lens`` cached tokens, or over the pages a route lists (row_ptr,
    col_idx from sa_route_pages): (o bf16 [B, 1, H, D], lse fp32 [B, H, 1] or
    None). H is a multiple of the cache's H_kv."""
    index = _cuda_index(q)
    if q.dim() != 4:
        raise ValueError("q must be [B, 1, H, D]")
    if o is None:
        o = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None and want_lse:
        lse = _empty((q.shape[0], q.shape[2], 1), torch.float32, q.device, stream)
    if workspace is None:
        p = make_cache_params(page_table, q=q, k_cache=k_cache, v_cache=v_cache)
        workspace = _empty((max(256, sa_attn_decode_workspace_bytes(p)),), torch.uint8, q.device,
                           stream)
    _call("sa_attn_decode", _bind().decode, index, stream, q, k_cache, v_cache, page_table,
          seq_lens, scale, row_ptr, col_idx, k_scale, v_scale, o, lse, workspace, dev_status)
    return o, lse


# ------------------------------------------------------------ drafted tokens --

def sa_attn_tree_workspace_bytes(p: sa_cache_params) -> int:
    return int(load_library().sa_attn_tree_workspace_bytes(ctypes.byref(p)))


def sa_attn_tree(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 page_table: torch.Tensor, seq_lens: torch.Tensor, scale: float = 0.0, *,
                 parents: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                 row_ptr: Optional[torch.Tensor] = None, col_idx: Optional[torch.Tensor] = None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 want_lse: bool = True, workspace: Optional[torch.Tensor] = None,
                 dev_status: Optional[torch.Tensor] = None, stream=None):
    """Attention of a tree of up to 64 new tokens of each sequence (q bf16 [B, S, H, D],
    appended behind its ``seq_lens`` tokens) over the cache: (o bf16 [B, S, H, D], lse
    fp32 [B, H, S] or None). Token s sees what was cached before, and the new tokens it
    continues: itself, ``parents``[b][s] (int32 [B, S], or [S] for one tree for all; -1:
    none), that one's parent, and so on; without ``parents`` every new token before it.
    ``new_lens``: how many of the S tokens each sequence has; rows of o and lse behind
    those are not written. ``row_ptr``, ``col_idx``: as in sa_attn_decode; pages with
    new tokens are attended whether listed or not. See sa.h."""
    index = _cuda_index(q)
    if q.dim() != 4:
        raise ValueError("q must be [B, S, H, D]")
    if o is None:
        o = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None and want_lse:
        lse = _empty((q.shape[0], q.shape[2], q.shape[1]), torch.float32, q.device, stream)
    if workspace is None:
        p = make_cache_params(page_table, q=q, k_cache=k_cache, v_cache=v_cache)
        workspace = _empty((max(256, sa_attn_tree_workspace_bytes(p)),), torch.uint8, q.device,
                           stream)
    _call("sa_attn_tree", _bind().tree, index, stream, q, k_cache, v_cache, page_table, seq_lens,
          scale, parents, new_lens, row_ptr, col_idx, k_scale, v_scale, o, lse, workspace,
          dev_status)
    return o, lse


def sa_cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                    seq_lens: torch.Tensor, path: torch.Tensor, path_lens: torch.Tensor, *,
                    k_sum: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                    lens_out: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """The new tokens of an accepted path move together behind each sequence's
    ``seq_lens`` tokens: token path[b][i] (int32 [B, S], ascending, i < path_lens[b]) to
    place i, keys and values. ``k_sum`` of the pages touched is made anew from the
    stored keys (``k_scale``: as in sa_cache_append), so path_lens = 0 takes all new
    tokens back; ``lens_out`` receives the new lengths."""
    index = _cuda_index(k_cache)
    _call("sa_cache_accept", _bind().accept, index, stream, k_cache, v_cache, page_table,
          seq_lens, path, path_lens, k_sum, k_scale, lens_out, dev_status)


# --------------------------------------------------------------------- pages --

def sa_pages_workspace_bytes(n_pages: int, rows: int) -> int:
    return int(load_library().sa_pages_workspace_bytes(int(n_pages), int(rows)))


def _pages_workspace(n_pages: int, rows: int, device, stream, workspace):
    if workspace is not None:
        return workspace
    return _empty((max(256, sa_pages_workspace_bytes(n_pages, rows)),), torch.uint8, device, stream)


def sa_pages_fork(page_table: torch.Tensor, seq_lens: torch.Tensor, refs: torch.Tensor,
                  src: torch.Tensor, *, table_out: Optional[torch.Tensor] = None,
                  lens_out: Optional[torch.Tensor] = None,
                  refs_out: Optional[torch.Tensor] = None,
                  moves: Optional[torch.Tensor] = None, n_moves: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None):
    """A new table whose sequence i continues sequence src[i] (int32 [N]; -1: an empty
    one) of the old one, which is given up: full pages are shared, the page in progress
    is copied for all but the first. refs int32 [n_pages] counts the places that hold a
    page (0: free). Returns (table_out [N, max_pages], lens_out [N], refs_out, moves
    int32 [N, 2], n_moves [1]): pass moves and n_moves to sa_cache_copy for each layer's
    caches. refs_out=refs counts in place."""
    index = _cuda_index(page_table)
    if any(t is None for t in (table_out, lens_out, refs_out, moves, n_moves, workspace)):
        for t, name, dim in ((page_table, "page_table", 2), (refs, "refs", 1), (src, "src", 1)):
            if not isinstance(t, torch.Tensor) or t.dim() != dim:
                raise ValueError(f"{name} must be int32 with {dim} dimension(s)")
        N, dev = src.shape[0], page_table.device
        new = lambda *shape: _empty(shape, torch.int32, dev, stream)
        table_out = new(N, page_table.shape[1]) if table_out is None else table_out
        lens_out = new(N) if lens_out is None else lens_out
        refs_out = new(refs.shape[0]) if refs_out is None else refs_out
        moves = new(N, 2) if moves is None else moves
        n_moves = new(1) if n_moves is None else n_moves
        workspace = _pages_workspace(refs.shape[0], max(N, page_table.shape[0]), dev, stream,
                                     workspace)
    _call("sa_pages_fork", _bind().fork, index, stream, page_table, seq_lens, refs, src, table_out,
          lens_out, refs_out, moves, n_moves, workspace, dev_status)
    return table_out, lens_out, refs_out, moves, n_moves


def sa_pages_resize(page_table: torch.Tensor, refs: torch.Tensor, seq_lens: torch.Tensor,
                    more: int = 0, *, more_lens: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Every sequence holds exactly the pages for seq_lens[b] + more tokens
    (``more_lens`` int32 [B] in place of ``more``): missing ones are taken from the free
    ones (refs 0), those behind are given back. Changes page_table and refs."""
    index = _cuda_index(page_table)
    if workspace is None:
        for t, name in ((page_table, "page_table"), (refs, "refs")):
            if not isinstance(t, torch.Tensor) or t.dim() < 1:
                raise ValueError(f"{name} must be an int32 tensor")
        workspace = _pages_workspace(refs.shape[0], page_table.shape[0], page_table.device, stream,
                                     None)
    _call("sa_pages_resize", _bind().resize, index, stream, page_table, refs, seq_lens, more,
          more_lens, workspace, dev_status)


def sa_pages_compact(page_table: Optional[torch.Tensor], refs: torch.Tensor, *,
                     table_out: Optional[torch.Tensor] = None,
                     refs_out: Optional[torch.Tensor] = None,
                     moves: Optional[torch.Tensor] = None,
                     n_moves: Optional[torch.Tensor] = None,
                     n_used: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    """The pages in use (refs > 0) move to the front of the pool. Returns (table_out,
    refs_out, moves int32 [n, 2], n_moves [1], n_used [1]): the table and counts by the
    new ids, the pairs (page, new id) for sa_cache_copy, how many pages are in use.
    table_out=page_table and refs_out=refs work in place."""
    index = _cuda_index(refs)
    if any(t is None for t in (table_out, refs_out, moves, n_moves, n_used, workspace)):
        new = lambda *shape: _empty(shape, torch.int32, refs.device, stream)
        rows = 1
        if page_table is not None:
            if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
                raise ValueError("page_table must be int32 [B, max_pages]")
            table_out = new(*page_table.shape) if table_out is None else table_out
            rows = page_table.shape[0]
        refs_out = new(refs.shape[0]) if refs_out is None else refs_out
        moves = new(max(1, refs.shape[0] // 2), 2) if moves is None else moves
        n_moves = new(1) if n_moves is None else n_moves
        n_used = new(1) if n_used is None else n_used
        workspace = _pages_workspace(refs.shape[0], rows, refs.device, stream, workspace)
    _call("sa_pages_compact", _bind().compact, index, stream, refs, page_table, table_out,
          refs_out, moves, n_moves, n_used, workspace, dev_status)
    return table_out, refs_out, moves, n_moves, n_used


def sa_cache_copy(k_cache: torch.Tensor, v_cache: torch.Tensor, moves: torch.Tensor,
                  n_moves: Optional[torch.Tensor] = None, *,
                  k_sum: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Page moves[i][0] to page moves[i][1] (int32 [n, 2]) for i < n_moves (int32 [1], all
    without): keys, values and, where given, key sums of one layer's caches."""
    index = _cuda_index(k_cache)
    _call("sa_cache_copy", _bind().copy, index, stream, k_cache, v_cache, moves, n_moves, k_sum,
          dev_status)


def check_dev_status(dev_status: torch.Tensor, what: str = "device status") -> None:
    """Raise if the kernels reported a device-side condition."""
    val = int(dev_status.item())
    if val:
        raise SaError(int(load_library().sa_dev_status_decode(val)), f"{what} (bits {val:#x})")
