"""ctypes binding of libveda.so (the C ABI in include/veda.h).

Argument marshalling only: every function here checks tensor devices, dtypes
and shapes, passes raw device pointers and the current CUDA stream to the
library function of the same name, and raises ``VedaError`` on a non-zero
status.  All computation runs in the library's CUDA kernels; there is no
fallback of any kind -- if the library is missing, importing this module
fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# VEDA_DEBUG_BOUNDS=1 loads the debug build (build.py --debug), whose kernels
# check every computed index and report a failed check as VEDA_ERR_BOUNDS.
LIB_PATH = os.path.join(_HERE, "libveda_debug.so" if os.environ.get("VEDA_DEBUG_BOUNDS") == "1" else "libveda.so")

VEDA_OK, VEDA_ERR_INVALID_ARG, VEDA_ERR_UNSUPPORTED, VEDA_ERR_CUDA, VEDA_ERR_TIMEOUT, VEDA_ERR_BOUNDS = range(6)
MAX_HEADS = 128
_STATUS_NAMES = {0: "VEDA_OK", 1: "VEDA_ERR_INVALID_ARG", 2: "VEDA_ERR_UNSUPPORTED", 3: "VEDA_ERR_CUDA",
                 4: "VEDA_ERR_TIMEOUT", 5: "VEDA_ERR_BOUNDS"}


class VedaError(RuntimeError):
    def __init__(self, status: int, func: str, message: str):
        super().__init__(f"{func}: {_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class veda_grid(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("W", ctypes.c_int32)]


class veda_tiling(ctypes.Structure):
    _fields_ = [("pt", ctypes.c_int32), ("ph", ctypes.c_int32), ("pw", ctypes.c_int32)]


class veda_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("heads", ctypes.c_int32), ("d", ctypes.c_int32), ("S", ctypes.c_int32),
                ("grid", veda_grid), ("tilings", ctypes.POINTER(veda_tiling))]


class veda_mlp(ctypes.Structure):
    _fields_ = [("w1", ctypes.c_void_p), ("b1", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("b2", ctypes.c_void_p),
                ("hidden", ctypes.c_int32), ("e", ctypes.c_int32)]


class veda_mlp_grad(ctypes.Structure):
    _fields_ = [("w1", ctypes.c_void_p), ("b1", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("b2", ctypes.c_void_p)]


class veda_rope(ctypes.Structure):
    tables, device = (), None     # make_rope: what the pointers point into, and where that is
    _fields_ = [("B", ctypes.c_int32), ("heads", ctypes.c_int32), ("d", ctypes.c_int32), ("grid", veda_grid),
                ("dim_t", ctypes.c_int32), ("dim_h", ctypes.c_int32), ("dim_w", ctypes.c_int32),
                ("table_t", ctypes.c_void_p), ("table_h", ctypes.c_void_p), ("table_w", ctypes.c_void_p),
                ("pairing", ctypes.c_int), ("norm", ctypes.c_int), ("eps", ctypes.c_float)]


class veda_tokens(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_n", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


_P = ctypes.POINTER(veda_problem)
_RP = ctypes.POINTER(veda_rope)
_TP = ctypes.POINTER(veda_tokens)
_I32, _I64, _F, _D, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
_V = ctypes.c_void_p
_I32P = ctypes.POINTER(ctypes.c_int32)
_SIG = {
    "veda_tile_layout": [_P, _I32P, _I32P],
    "veda_keep_count": [_P, ctypes.c_float, _I32P, _I32P],
    "veda_tile_permute": [_P, _V, _V, _V],
    "veda_tile_unpermute": [_P, _V, _V, _V],
    "veda_tile_permute_tripool": [_P, _V, _V, _V, _V],
    "veda_tripool": [_P, _V, _V, _V],
    "veda_tripool_grid": [_P, _V, _V, _V],
    "veda_score_topk_workspace": [_P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
    "veda_tile_score_topk": [_P, _V, _V, ctypes.POINTER(veda_mlp), ctypes.POINTER(veda_mlp), ctypes.c_float, _V,
                             ctypes.c_int32, _V, _V, ctypes.c_size_t, _V],
    "veda_tile_score_topk_noalloc": [_P, _V, _V, ctypes.POINTER(veda_mlp), ctypes.POINTER(veda_mlp), ctypes.c_float,
                                     _V, ctypes.c_int32, _V, _V],
    "veda_tile_sparse_attn": [_P, _V, _V, _V, _V, ctypes.c_int32, ctypes.c_float, _V, _V, _V],
    "veda_tile_sparse_attn_grid": [_P, _V, _V, _V, _V, ctypes.c_int32, ctypes.c_float, _V, _V, _V],
    "veda_attn_config": [_P, ctypes.c_int32, _I32P, _I32P, ctypes.POINTER(ctypes.c_size_t)],
    "veda_tile_map_workspace": [_P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
    "veda_tile_map_maxpool": [_P, _V, _V, _V, ctypes.c_int32, ctypes.c_float, _V, _V, ctypes.c_size_t, _V],
    "veda_tile_map_maxpool_grid": [_P, _V, _V, _V, ctypes.c_int32, ctypes.c_float, _V, _V, ctypes.c_size_t, _V],
    "veda_distill_workspace": [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
    "veda_distill_loss_grad": [_P, _V, _V, ctypes.POINTER(veda_mlp), ctypes.POINTER(veda_mlp), _V, _V, ctypes.c_int32,
                               _V, ctypes.POINTER(veda_mlp_grad), ctypes.POINTER(veda_mlp_grad), _V, ctypes.c_size_t,
                               _V],
    "veda_head_error": [_P, _V, _V, _V, _V, _V, ctypes.c_size_t, _V],
    "veda_attn_backward_workspace": [_P, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)],
    "veda_tile_sparse_attn_backward_grid": [_P, _V, _V, _V, _V, _V, _V, _V, ctypes.c_int32, ctypes.c_float, _V, _V,
                                            _V, _V, ctypes.c_size_t, _V],
    "veda_add_rms_norm": [_I64, _I32, _I32, _V, _I64, _I32, _V, _I64, _V, _F, _V, _V, _V],
    "veda_add_rms_norm_fp8": [_I64, _I32, _I32, _V, _I64, _I32, _V, _I64, _V, _F, _V, _V, _V, _V],
    "veda_add_rms_norm_backward_workspace": [_I64, _I32, ctypes.POINTER(_SZ)],
    "veda_add_rms_norm_backward": [_I64, _I32, _I32, _V, _I32, _V, _V, _V, _F, _V, _V, _V, _V, _SZ, _V],
    "veda_quant_fp8": [_I32, _I64, _I32, _I32, _I32, _V, _I64, _I64, _I64, _V, _V, _V],
    "veda_quant_fp8_weight": [_I32, _I32, _I32, _V, _V, _V, _V],
    "veda_gemm_fp8": [_I32, _I32, _I32, _V, _I64, _V, _V, _I64, _V, _V, _I32, _V, _I64, _V],
    "veda_rope_table": [_I32, _I32, _D, _D, _D, _V, _V],
    "veda_qkv_norm_rope": [_RP, _I32, _TP, _TP, _TP, _V, _V, _V, _V, _V, _V],
    "veda_qkv_norm_rope_backward_workspace": [_RP, ctypes.POINTER(_SZ)],
    "veda_qkv_norm_rope_backward": [_RP, _I32, _TP, _TP, _V, _V, _V, _V, _V, _TP, _TP, _TP, _V, _V, _V, _SZ, _V],
    "veda_sync_status": [_V],
    "veda_set_wait_timeout_ns": [ctypes.c_uint64],
    "veda_selftest_wait_timeout": [ctypes.c_uint64, _V],
    "veda_selftest_bounds": [_V],
    "veda_bounds_checked": [],
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); "
                          "run tile_sparse_attention_head_b200/build.py" +
                          (" --debug" if LIB_PATH.endswith("_debug.so") else ""))
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in _SIG.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.veda_last_error.restype = ctypes.c_char_p
    lib.veda_last_error.argtypes = []
    lib.veda_version.restype = ctypes.c_char_p
    lib.veda_version.argtypes = []
    return lib


LIB = _load()


def _check(status: int, func: str) -> None:
    if status != VEDA_OK:
        raise VedaError(status, func, LIB.veda_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor], name: str, dtype: Optional[torch.dtype] = None,
         shape: Optional[Tuple[int, ...]] = None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t.data_ptr()


class Problem:
    """The problem statement (B, heads, d, S, grid, per-head tilings) as the C struct."""

    def __init__(self, B: int, heads: int, d: int, S: int, grid: Sequence[int],
                 tilings: Sequence[Sequence[int]]):
        self.B, self.heads, self.d, self.S = int(B), int(heads), int(d), int(S)
        self.grid = tuple(int(v) for v in grid)
        self.tilings = tuple(tuple(int(v) for v in t) for t in tilings)
        if len(self.tilings) != self.heads:
            raise ValueError("one tiling per head is required")
        self._tilings_arr = (veda_tiling * max(1, self.heads))(*[veda_tiling(*t) for t in self.tilings])
        self.c = veda_problem(self.B, self.heads, self.d, self.S, veda_grid(*self.grid),
                              ctypes.cast(self._tilings_arr, ctypes.POINTER(veda_tiling)))
        nts = (ctypes.c_int32 * self.heads)()
        ntmax = ctypes.c_int32()
        _check(LIB.veda_tile_layout(ctypes.byref(self.c), nts, ctypes.byref(ntmax)), "veda_tile_layout")
        self.nt_per_head = list(nts)
        self.nt_max = int(ntmax.value)

    @property
    def N(self) -> int:
        return self.grid[0] * self.grid[1] * self.grid[2]

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def grid_shape(self) -> Tuple[int, int, int, int]:
        return (self.B, self.heads, self.N, self.d)

    def tile_shape(self) -> Tuple[int, int, int, int]:
        return (self.B, self.heads, self.nt_max * self.S, self.d)

    def keep_count(self, keep_ratio: float):
        ks = (ctypes.c_int32 * self.heads)()
        kmax = ctypes.c_int32()
        _check(LIB.veda_keep_count(self.ref, ctypes.c_float(keep_ratio), ks, ctypes.byref(kmax)), "veda_keep_count")
        return list(ks), int(kmax.value)


def veda_tile_permute(p: Problem, x: torch.Tensor, xp: torch.Tensor, stream=None) -> torch.Tensor:
    _check(LIB.veda_tile_permute(p.ref, _ptr(x, "x", torch.bfloat16, p.grid_shape()),
                                 _ptr(xp, "xp", torch.bfloat16, p.tile_shape()), _stream(stream)),
           "veda_tile_permute")
    return xp


def veda_tile_permute_tripool(p: Problem, x: torch.Tensor, xp: torch.Tensor, desc: torch.Tensor,
                              stream=None) -> torch.Tensor:
    _check(LIB.veda_tile_permute_tripool(p.ref, _ptr(x, "x", torch.bfloat16, p.grid_shape()),
                                         _ptr(xp, "xp", torch.bfloat16, p.tile_shape()),
                                         _ptr(desc, "desc", torch.float32, (p.B, p.heads, p.nt_max, 3 * p.d)),
                                         _stream(stream)), "veda_tile_permute_tripool")
    return xp


def veda_tile_unpermute(p: Problem, xp: torch.Tensor, x: torch.Tensor, stream=None) -> torch.Tensor:
    _check(LIB.veda_tile_unpermute(p.ref, _ptr(xp, "xp", torch.bfloat16, p.tile_shape()),
                                   _ptr(x, "x", torch.bfloat16, p.grid_shape()), _stream(stream)),
           "veda_tile_unpermute")
    return x


def veda_tripool(p: Problem, xp: torch.Tensor, desc: torch.Tensor, stream=None) -> torch.Tensor:
    _check(LIB.veda_tripool(p.ref, _ptr(xp, "xp", torch.bfloat16, p.tile_shape()),
                            _ptr(desc, "desc", torch.float32, (p.B, p.heads, p.nt_max, 3 * p.d)), _stream(stream)),
           "veda_tripool")
    return desc


def veda_tripool_grid(p: Problem, x: torch.Tensor, desc: torch.Tensor, stream=None) -> torch.Tensor:
    _check(LIB.veda_tripool_grid(p.ref, _ptr(x, "x", torch.bfloat16, p.grid_shape()),
                                 _ptr(desc, "desc", torch.float32, (p.B, p.heads, p.nt_max, 3 * p.d)),
                                 _stream(stream)),
           "veda_tripool_grid")
    return desc


def veda_score_topk_workspace(p: Problem, e: int) -> int:
    n = ctypes.c_size_t()
    _check(LIB.veda_score_topk_workspace(p.ref, int(e), ctypes.byref(n)), "veda_score_topk_workspace")
    return int(n.value)


def make_mlp(w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, b2: torch.Tensor) -> veda_mlp:
    """C struct for one set of per-head estimator weights (fp32 device tensors)."""
    heads, hidden, _ = w1.shape
    e = w2.shape[1]
    for t, n in ((w1, "w1"), (b1, "b1"), (w2, "w2"), (b2, "b2")):
        _ptr(t, n, torch.float32)
    if tuple(b1.shape) != (heads, hidden) or tuple(w2.shape) != (heads, e, hidden) or tuple(b2.shape) != (heads, e):
        raise ValueError("estimator weight shapes must be w1 [h,hid,3d], b1 [h,hid], w2 [h,e,hid], b2 [h,e]")
    return veda_mlp(w1.data_ptr(), b1.data_ptr(), w2.data_ptr(), b2.data_ptr(), int(hidden), int(e))


def veda_tile_score_topk(p: Problem, desc_q: torch.Tensor, desc_k: torch.Tensor, mlp_q: veda_mlp, mlp_k: veda_mlp,
                         keep_ratio: float, idx: torch.Tensor, probs: Optional[torch.Tensor],
                         workspace: torch.Tensor, stream=None) -> torch.Tensor:
    dshape = (p.B, p.heads, p.nt_max, 3 * p.d)
    k_max = int(idx.shape[-1])
    _check(LIB.veda_tile_score_topk(
        p.ref, _ptr(desc_q, "desc_q", torch.float32, dshape), _ptr(desc_k, "desc_k", torch.float32, dshape),
        ctypes.byref(mlp_q), ctypes.byref(mlp_k), ctypes.c_float(keep_ratio),
        _ptr(idx, "idx", torch.int32, (p.B, p.heads, p.nt_max, k_max)), k_max,
        _ptr(probs, "probs", torch.float32, (p.B, p.heads, p.nt_max, p.nt_max)),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream)),
        "veda_tile_score_topk")
    return idx


def veda_tile_score_topk_noalloc(p: Problem, desc_q: torch.Tensor, desc_k: torch.Tensor, mlp_q: veda_mlp,
                                 mlp_k: veda_mlp, keep_ratio: float, idx: torch.Tensor,
                                 probs: Optional[torch.Tensor], stream=None) -> torch.Tensor:
    """veda_tile_score_topk without a workspace, for callers that cannot allocate device scratch."""
    dshape = (p.B, p.heads, p.nt_max, 3 * p.d)
    k_max = int(idx.shape[-1])
    _check(LIB.veda_tile_score_topk_noalloc(
        p.ref, _ptr(desc_q, "desc_q", torch.float32, dshape), _ptr(desc_k, "desc_k", torch.float32, dshape),
        ctypes.byref(mlp_q), ctypes.byref(mlp_k), ctypes.c_float(keep_ratio),
        _ptr(idx, "idx", torch.int32, (p.B, p.heads, p.nt_max, k_max)), k_max,
        _ptr(probs, "probs", torch.float32, (p.B, p.heads, p.nt_max, p.nt_max)), _stream(stream)),
        "veda_tile_score_topk_noalloc")
    return idx


def veda_tile_sparse_attn(p: Problem, qp: torch.Tensor, kp: torch.Tensor, vp: torch.Tensor, idx: torch.Tensor,
                          op: torch.Tensor, lse: Optional[torch.Tensor] = None, scale: float = 0.0,
                          stream=None) -> torch.Tensor:
    ts = p.tile_shape()
    k_max = int(idx.shape[-1])
    _check(LIB.veda_tile_sparse_attn(
        p.ref, _ptr(qp, "qp", torch.bfloat16, ts), _ptr(kp, "kp", torch.bfloat16, ts),
        _ptr(vp, "vp", torch.bfloat16, ts), _ptr(idx, "idx", torch.int32, (p.B, p.heads, p.nt_max, k_max)), k_max,
        ctypes.c_float(scale), _ptr(op, "op", torch.bfloat16, ts),
        _ptr(lse, "lse", torch.float32, (p.B, p.heads, p.nt_max * p.S)), _stream(stream)),
        "veda_tile_sparse_attn")
    return op


def veda_tile_sparse_attn_grid(p: Problem, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor,
                               o: torch.Tensor, lse: Optional[torch.Tensor] = None, scale: float = 0.0,
                               stream=None) -> torch.Tensor:
    gs = p.grid_shape()
    k_max = int(idx.shape[-1])
    _check(LIB.veda_tile_sparse_attn_grid(
        p.ref, _ptr(q, "q", torch.bfloat16, gs), _ptr(k, "k", torch.bfloat16, gs),
        _ptr(v, "v", torch.bfloat16, gs), _ptr(idx, "idx", torch.int32, (p.B, p.heads, p.nt_max, k_max)), k_max,
        ctypes.c_float(scale), _ptr(o, "o", torch.bfloat16, gs),
        _ptr(lse, "lse", torch.float32, (p.B, p.heads, p.N)), _stream(stream)),
        "veda_tile_sparse_attn_grid")
    return o


def veda_attn_backward_workspace(p: Problem, k_max: int) -> int:
    n = ctypes.c_size_t()
    _check(LIB.veda_attn_backward_workspace(p.ref, int(k_max), ctypes.byref(n)), "veda_attn_backward_workspace")
    return int(n.value)


def veda_tile_sparse_attn_backward_grid(p: Problem, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                        o: torch.Tensor, lse: torch.Tensor, d_o: torch.Tensor, idx: torch.Tensor,
                                        dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                                        workspace: torch.Tensor, scale: float = 0.0, stream=None):
    """dq, dk, dv of veda_tile_sparse_attn_grid for the upstream gradient d_o (all grid order)."""
    gs = p.grid_shape()
    k_max = int(idx.shape[-1])
    _check(LIB.veda_tile_sparse_attn_backward_grid(
        p.ref, _ptr(q, "q", torch.bfloat16, gs), _ptr(k, "k", torch.bfloat16, gs), _ptr(v, "v", torch.bfloat16, gs),
        _ptr(o, "o", torch.bfloat16, gs), _ptr(lse, "lse", torch.float32, (p.B, p.heads, p.N)),
        _ptr(d_o, "d_o", torch.bfloat16, gs), _ptr(idx, "idx", torch.int32, (p.B, p.heads, p.nt_max, k_max)), k_max,
        ctypes.c_float(scale), _ptr(dq, "dq", torch.bfloat16, gs), _ptr(dk, "dk", torch.bfloat16, gs),
        _ptr(dv, "dv", torch.bfloat16, gs), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "veda_tile_sparse_attn_backward_grid")
    return dq, dk, dv


def veda_attn_config(p: Problem, k_max: int) -> Tuple[int, int, int]:
    """(K ring depth, V ring depth, dynamic shared memory bytes) of the attention launch."""
    ks, vs, nb = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_size_t()
    _check(LIB.veda_attn_config(p.ref, int(k_max), ctypes.byref(ks), ctypes.byref(vs), ctypes.byref(nb)),
           "veda_attn_config")
    return int(ks.value), int(vs.value), int(nb.value)


def veda_tile_map_workspace(p: Problem, R: int) -> int:
    n = ctypes.c_size_t()
    _check(LIB.veda_tile_map_workspace(p.ref, int(R), ctypes.byref(n)), "veda_tile_map_workspace")
    return int(n.value)


def veda_tile_map_maxpool(p: Problem, qp: torch.Tensor, kp: torch.Tensor, rows: torch.Tensor, out: torch.Tensor,
                          workspace: torch.Tensor, scale: float = 0.0, stream=None) -> torch.Tensor:
    ts = p.tile_shape()
    R = int(rows.shape[-1])
    _check(LIB.veda_tile_map_maxpool(
        p.ref, _ptr(qp, "qp", torch.bfloat16, ts), _ptr(kp, "kp", torch.bfloat16, ts),
        _ptr(rows, "rows", torch.int32, (p.B * p.heads, R)), R, ctypes.c_float(scale),
        _ptr(out, "map", torch.float32, (p.B, p.heads, R, p.nt_max)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "veda_tile_map_maxpool")
    return out


def veda_tile_map_maxpool_grid(p: Problem, q: torch.Tensor, k: torch.Tensor, rows: torch.Tensor, out: torch.Tensor,
                               workspace: torch.Tensor, scale: float = 0.0, stream=None) -> torch.Tensor:
    """The max-pooled tile map from grid-order q, k [B, heads, N, d] bf16 (no tile-major copies)."""
    gs = p.grid_shape()
    R = int(rows.shape[-1])
    _check(LIB.veda_tile_map_maxpool_grid(
        p.ref, _ptr(q, "q", torch.bfloat16, gs), _ptr(k, "k", torch.bfloat16, gs),
        _ptr(rows, "rows", torch.int32, (p.B * p.heads, R)), R, ctypes.c_float(scale),
        _ptr(out, "map", torch.float32, (p.B, p.heads, R, p.nt_max)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "veda_tile_map_maxpool_grid")
    return out


def veda_distill_workspace(p: Problem, hidden: int, e: int, R: int) -> int:
    n = ctypes.c_size_t()
    _check(LIB.veda_distill_workspace(p.ref, int(hidden), int(e), int(R), ctypes.byref(n)), "veda_distill_workspace")
    return int(n.value)


def make_mlp_grad(w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, b2: torch.Tensor) -> veda_mlp_grad:
    """C struct of gradient outputs for one estimator (fp32 device tensors shaped like its weights)."""
    for t, n in ((w1, "w1"), (b1, "b1"), (w2, "w2"), (b2, "b2")):
        _ptr(t, n, torch.float32)
    return veda_mlp_grad(w1.data_ptr(), b1.data_ptr(), w2.data_ptr(), b2.data_ptr())


def veda_distill_loss_grad(p: Problem, desc_q: torch.Tensor, desc_k: torch.Tensor, mlp_q: veda_mlp, mlp_k: veda_mlp,
                           tile_map: torch.Tensor, rows: torch.Tensor, loss: torch.Tensor, grad_q: veda_mlp_grad,
                           grad_k: veda_mlp_grad, workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Row-wise KL distillation loss of the estimator against the tile map, and its gradients."""
    dshape = (p.B, p.heads, p.nt_max, 3 * p.d)
    R = int(rows.shape[-1])
    _check(LIB.veda_distill_loss_grad(
        p.ref, _ptr(desc_q, "desc_q", torch.float32, dshape), _ptr(desc_k, "desc_k", torch.float32, dshape),
        ctypes.byref(mlp_q), ctypes.byref(mlp_k),
        _ptr(tile_map, "map", torch.float32, (p.B, p.heads, R, p.nt_max)),
        _ptr(rows, "rows", torch.int32, (p.B * p.heads, R)), R, _ptr(loss, "loss", torch.float32, (1,)),
        ctypes.byref(grad_q), ctypes.byref(grad_k), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _stream(stream)), "veda_distill_loss_grad")
    return loss


def veda_head_error(p: Problem, o: torch.Tensor, o_ref: torch.Tensor, err: torch.Tensor, ref_sq: torch.Tensor,
                    workspace: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-head sums of (o - o_ref)^2 and o_ref^2 over grid-order bf16 outputs."""
    gs = p.grid_shape()
    _check(LIB.veda_head_error(p.ref, _ptr(o, "o", torch.bfloat16, gs), _ptr(o_ref, "o_ref", torch.bfloat16, gs),
                               _ptr(err, "err", torch.float32, (p.heads,)),
                               _ptr(ref_sq, "ref_sq", torch.float32, (p.heads,)), _ptr(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(), _stream(stream)), "veda_head_error")
    return err, ref_sq


# ---------------------------------------------------------------- around the attention
#
# These take tensors of any device: the call runs on its tensors' device (all on
# one) and, without a `stream`, on that device's current stream.  A call on one
# token takes a few microseconds on the GPU, so what runs on the host around it
# is kept short: device, stream and shape are compared as plain integers and
# tuples, and messages are put together only when something is refused.

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_NORMS = {"none": 0, "row": 1, "head": 2}
_PAIRINGS = {"interleaved": 0, "halves": 1}
FP8 = torch.float8_e4m3fn
_F32 = torch.float32


def _type(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32 (got {t.dtype})")
    return code


def _device(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _at(t: Optional[torch.Tensor], name: str, dev: int, dtype: torch.dtype, shape: Tuple[int, ...]) -> Optional[int]:
    """Pointer of a dense tensor of this device, type and shape."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the first operand on cuda:{dev}" if t.is_cuda
                         else f"{name} must be a CUDA tensor")
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _ptr(t, name, dtype, shape)      # says what is wrong
    return t.data_ptr()


def _rows(t: Optional[torch.Tensor], name: str, dev: int, shape=None) -> Tuple[Optional[int], int]:
    """Pointer and row stride of a [rows, C] tensor whose channels are contiguous."""
    if t is None:
        return None, 0
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the first operand on cuda:{dev}" if t.is_cuda
                         else f"{name} must be a CUDA tensor")
    size = t.shape
    if len(size) != 2 or (size[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, C] with contiguous channels")
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(size)})")
    return t.data_ptr(), t.stride(0) if size[0] > 1 else size[1]


def _too_large(*sizes: int) -> None:
    """Refuses sizes that the library's 32-bit arguments cannot hold (ctypes would pass their low 32 bits)."""
    raise ValueError(f"a size in {sizes} does not fit 32 bits")


def _call(func: str, dev: int, stream, *args) -> None:
    """Runs the library function with `dev` current, on `stream` or that device's current stream."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _call(func, dev, stream, *args)
    status = getattr(LIB, func)(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status != VEDA_OK:
        _check(status, func)


def _on_device(device, fn):
    """fn() with `device` (None: the current one) current: the workspace sizes depend on it."""
    if device is None or device == torch._C._cuda_getDevice():
        return fn()
    with torch.cuda.device(device):
        return fn()


def veda_add_rms_norm(x: torch.Tensor, delta: Optional[torch.Tensor], weight: torch.Tensor, eps: float,
                      h: Optional[torch.Tensor], y: torch.Tensor, stream=None) -> torch.Tensor:
    """h = x + delta and its RMS norm y, [rows, C]; y is of delta's type (x's without a delta)."""
    dev, shape = _device(x, "x"), x.shape
    xp, ldx = _rows(x, "x", dev)
    if shape[1] >> 31:
        _too_large(shape[1])
    dp, ldd = _rows(delta, "delta", dev, shape)
    td = y.dtype if delta is None else delta.dtype
    _call("veda_add_rms_norm", dev, stream, shape[0], shape[1], _type(x, "x"), xp, ldx,
          _type(y, "y") if delta is None else _type(delta, "delta"), dp, ldd, _at(weight, "weight", dev, _F32, shape[1:]),
          eps, _at(h, "h", dev, x.dtype, shape), _at(y, "y", dev, td, shape))
    return y


def veda_add_rms_norm_fp8(x: torch.Tensor, delta: Optional[torch.Tensor], weight: torch.Tensor, eps: float,
                          h: Optional[torch.Tensor], y8: torch.Tensor, y_scale: torch.Tensor,
                          stream=None) -> torch.Tensor:
    """veda_add_rms_norm with y in e4m3 and a scale per row and 128 channels, [ceil(C/128), rows]."""
    dev, shape = _device(x, "x"), x.shape
    xp, ldx = _rows(x, "x", dev)
    dp, ldd = _rows(delta, "delta", dev, shape)
    rows, C = shape
    if C >> 31:
        _too_large(C)
    tx = _type(x, "x")
    _call("veda_add_rms_norm_fp8", dev, stream, rows, C, tx, xp, ldx,
          tx if delta is None else _type(delta, "delta"), dp, ldd, _at(weight, "weight", dev, _F32, (C,)), eps,
          _at(h, "h", dev, x.dtype, shape), _at(y8, "y8", dev, FP8, shape),
          _at(y_scale, "y_scale", dev, _F32, ((C + 127) // 128, rows)))
    return y8


# The three below run the same library functions for layer.py, on tensors that
# it has laid out or made itself (rows, and outputs of the right shape on the
# right device): only what comes from the caller unseen is checked.

def _layer_norm_forward(x, delta, weight, eps, h, y, scale) -> None:
    dev = x.get_device()
    rows, C = x.shape
    tx = _DTYPES.get(x.dtype)
    if dev < 0 or tx is None or C >> 31:
        _device(x, "x"), _type(x, "x"), _too_large(C)
    if delta is None:
        td, dp, ldd = tx, None, 0
    else:
        if delta.get_device() != dev:
            _rows(delta, "delta", dev)
        td, dp, ldd = _type(delta, "delta"), delta.data_ptr(), delta.stride(0) if rows > 1 else C
    args = (rows, C, tx, x.data_ptr(), x.stride(0) if rows > 1 else C, td, dp, ldd,
            _at(weight, "weight", dev, _F32, (C,)), eps, None if h is None else h.data_ptr(), y.data_ptr())
    if scale is None:
        _call("veda_add_rms_norm", dev, None, *args)
    else:
        _call("veda_add_rms_norm_fp8", dev, None, *args, scale.data_ptr())


def _layer_norm_backward(h, dy, dh, weight, eps, dx, ddelta, dweight) -> None:
    dev = h.get_device()
    rows, C = h.shape
    ws, size = None, 0
    if dweight is not None:
        size = veda_add_rms_norm_backward_workspace(rows, C, dev)
        ws = h.new_empty(size, dtype=torch.uint8)
    _call("veda_add_rms_norm_backward", dev, None, rows, C, _DTYPES[h.dtype], h.data_ptr(), _type(dy, "dy"), dy.data_ptr(),
          None if dh is None else dh.data_ptr(), weight.data_ptr(), eps,
          None if dx is None else dx.data_ptr(), None if ddelta is None else ddelta.data_ptr(),
          None if dweight is None else dweight.data_ptr(), None if ws is None else ws.data_ptr(), size)


def _layer_gemm(a, a_scale, b, b_scale, bias, out_dtype) -> torch.Tensor:
    dev = _device(a, "a")
    ap, lda = _rows(a, "a", dev)
    bp, ldb = _rows(b, "b", dev)
    (M, K), (N, Kb) = a.shape, b.shape
    if a.dtype is not FP8 or b.dtype is not FP8 or Kb != K:
        raise ValueError(f"a and b must be {FP8} [M, K] and [N, K] (got {a.dtype} {tuple(a.shape)}, {b.dtype} {tuple(b.shape)})")
    if (M | N | K) >> 31:
        _too_large(M, N, K)
    kb = (K + 127) // 128
    out = a.new_empty((M, N), dtype=out_dtype)
    _call("veda_gemm_fp8", dev, None, M, N, K, ap, lda, _at(a_scale, "a_scale", dev, _F32, (kb, M)), bp, ldb,
          _at(b_scale, "b_scale", dev, _F32, ((N + 127) // 128, kb)), _at(bias, "bias", dev, _F32, (N,)),
          _type(out, "out"), out.data_ptr(), N)
    return out


def veda_add_rms_norm_backward_workspace(rows: int, C: int, device=None) -> int:
    n = _SZ()
    if C >> 31:
        _too_large(C)
    if device is not None and device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return veda_add_rms_norm_backward_workspace(rows, C)
    _check(LIB.veda_add_rms_norm_backward_workspace(rows, C, ctypes.byref(n)), "veda_add_rms_norm_backward_workspace")
    return n.value


def veda_add_rms_norm_backward(h: torch.Tensor, dy: torch.Tensor, dh: Optional[torch.Tensor], weight: torch.Tensor,
                               eps: float, dx: Optional[torch.Tensor], ddelta: Optional[torch.Tensor],
                               dweight: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                               stream=None) -> None:
    """Gradients of veda_add_rms_norm: dx in h's type, ddelta in dy's type, dweight fp32; None leaves one out."""
    dev, shape = _device(h, "h"), h.shape
    if len(shape) != 2:
        raise ValueError("h must be [rows, C]")
    if shape[1] >> 31:
        _too_large(shape[1])
    th, td = h.dtype, dy.dtype
    _call("veda_add_rms_norm_backward", dev, stream, shape[0], shape[1], _type(h, "h"), _at(h, "h", dev, th, shape),
          _type(dy, "dy"), _at(dy, "dy", dev, td, shape), _at(dh, "dh", dev, th, shape),
          _at(weight, "weight", dev, _F32, shape[1:]), eps,
          _at(dx, "dx", dev, th, shape), _at(ddelta, "ddelta", dev, td, shape),
          _at(dweight, "dweight", dev, _F32, shape[1:]), *_scratch(workspace, dev))


def _scratch(workspace: Optional[torch.Tensor], dev: int) -> Tuple[Optional[int], int]:
    if workspace is None:
        return None, 0
    return _at(workspace, "workspace", dev, workspace.dtype, workspace.shape), workspace.numel() * workspace.element_size()


def veda_quant_fp8(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, stream=None) -> torch.Tensor:
    """[rows, C], or the attention's grid-order [B, heads, N, d], to e4m3 rows [rows, C] (B*N rows of heads*d
    channels) and scales [ceil(C/128), rows].  Channels contiguous, other strides free multiples of 8."""
    dev = _device(x, "x")
    if x.dim() == 2:
        (N, d), (sn, sd) = x.shape, x.stride()
        B, heads, sb, sh = 1, 1, 0, 0
    elif x.dim() == 4:
        (B, heads, N, d), (sb, sh, sn, sd) = x.shape, x.stride()
    else:
        raise ValueError("x must be [rows, C] or [B, heads, N, d]")
    if d > 1 and sd != 1:
        raise ValueError("the channels of x must be contiguous")
    if (B | heads | d) >> 31:
        _too_large(B, heads, d)
    rows, C = B * N, heads * d
    _call("veda_quant_fp8", dev, stream, B, N, heads, d, _type(x, "x"), x.data_ptr(),
          sb if B > 1 else 0, sn if N > 1 else 0, sh if heads > 1 else 0,
          _at(q, "q", dev, FP8, (rows, C)), _at(scale, "scale", dev, _F32, ((C + 127) // 128, rows)))
    return q


def veda_quant_fp8_weight(w: torch.Tensor, q: torch.Tensor, scale: torch.Tensor, stream=None) -> torch.Tensor:
    """A weight [N, K] to e4m3 with a scale per 128 x 128 block, [ceil(N/128), ceil(K/128)]."""
    dev = _device(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    N, K = w.shape
    if (N | K) >> 31:
        _too_large(N, K)
    _call("veda_quant_fp8_weight", dev, stream, N, K, _type(w, "w"), _at(w, "w", dev, w.dtype, (N, K)),
          _at(q, "q", dev, FP8, (N, K)), _at(scale, "scale", dev, _F32, ((N + 127) // 128, (K + 127) // 128)))
    return q


def veda_gemm_fp8(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
                  bias: Optional[torch.Tensor], out: torch.Tensor, stream=None) -> torch.Tensor:
    """out [M, N] = a [M, K] b [N, K]^T (+ bias) of e4m3 operands with a scale per row and 128 channels of a,
    [ceil(K/128), M], and per 128 x 128 block of b, [ceil(N/128), ceil(K/128)]; out bf16 or fp32."""
    dev = _device(a, "a")
    ap, lda = _rows(a, "a", dev)
    bp, ldb = _rows(b, "b", dev)
    (M, K), N = a.shape, b.shape[0]
    if a.dtype is not FP8 or b.dtype is not FP8:
        raise ValueError(f"a and b must be {FP8} (got {a.dtype} and {b.dtype})")
    if b.shape[1] != K:
        raise ValueError(f"b must be [N, {K}] (got {tuple(b.shape)})")
    if (M | N | K) >> 31:
        _too_large(M, N, K)
    op, ldo = _rows(out, "out", dev, (M, N))
    kb = (K + 127) // 128
    _call("veda_gemm_fp8", dev, stream, M, N, K, ap, lda, _at(a_scale, "a_scale", dev, _F32, (kb, M)), bp, ldb,
          _at(b_scale, "b_scale", dev, _F32, ((N + 127) // 128, kb)), _at(bias, "bias", dev, _F32, (N,)),
          _type(out, "out"), op, ldo)
    return out


def veda_rope_table(table: torch.Tensor, theta: float = 10000.0, start: float = 0.0, step: float = 1.0,
                    stream=None) -> torch.Tensor:
    """(cos, sin) of (start + step*i) * theta^(-2j/dim) into table [n, dim/2, 2] fp32 (angles in fp64)."""
    dev = _device(table, "table")
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be [n, dim/2, 2]")
    if (table.shape[0] | 2 * table.shape[1]) >> 31:
        _too_large(*table.shape)
    _call("veda_rope_table", dev, stream, table.shape[0], 2 * table.shape[1], theta, start, step,
          _at(table, "table", dev, _F32, table.shape))
    return table


def make_rope(B: int, heads: int, d: int, grid: Sequence[int], tables: Sequence[Optional[torch.Tensor]],
              pairing: str = "interleaved", norm: str = "row", eps: float = 1e-6) -> veda_rope:
    """C struct of a rotary description; tables (time, height, width): fp32 [at least the grid's size, pairs, 2]
    device tensors of one device, or None for an axis without channels.  The struct keeps them alive."""
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)} (got {norm!r})")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(_PAIRINGS)} (got {pairing!r})")
    if len(grid) != 3 or len(tables) != 3:
        raise ValueError("grid and tables have three entries: time, height, width")
    dims, ptrs, dev = [], [], None
    for t, n in zip(tables, grid):
        if t is None:
            dims.append(0)
            ptrs.append(None)
            continue
        shape = t.shape
        if len(shape) != 3 or shape[2] != 2 or shape[0] < n:
            raise ValueError(f"a table must be [at least {n}, pairs, 2] (got {tuple(shape)})")
        dims.append(2 * shape[1])
        dev = _device(t, "a table") if dev is None else dev
        ptrs.append(_at(t, "a table", dev, _F32, shape) if shape[1] else None)
    T, H, W = map(int, grid)
    if min(T, H, W) < 1:      # also what would be a valid size in its low 32 bits
        raise ValueError(f"grid dimensions must be >= 1 (got {T} x {H} x {W})")
    if max(B, heads, d, T, H, W, *dims) >> 31:
        _too_large(B, heads, d, T, H, W, *dims)
    r = veda_rope(B, heads, d, veda_grid(T, H, W), *dims, *ptrs, _PAIRINGS[pairing], _NORMS[norm], eps)
    r.tables, r.device = tuple(tables), dev
    return r


def _same_device(r: veda_rope, dev: int) -> None:
    if r.device is not None and r.device != dev:
        raise ValueError(f"the tables are on cuda:{r.device}, the operands on cuda:{dev}")


def _tokens(t: Optional[torch.Tensor], r: veda_rope, name: str, dev: int, dtype: torch.dtype, shape):
    """A token-order operand as the C struct's reference; shape: its [B, N, heads, d]."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the first operand on cuda:{dev}" if t.is_cuda
                         else f"{name} must be a CUDA tensor")
    sb, sn, sh, sc = t.stride() if t.dim() == 4 else (0, 0, 0, 0)
    if t.shape != shape or sc != 1 or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)} with contiguous channels (got {t.dtype} {tuple(t.shape)})")
    return ctypes.byref(veda_tokens(t.data_ptr(), sb if shape[0] > 1 else 0, sn if shape[1] > 1 else 0,
                                    sh if shape[2] > 1 else 0))


def _norm_weight(w: Optional[torch.Tensor], r: veda_rope, name: str, dev: int) -> Optional[int]:
    if w is None or r.norm == 0:
        return None
    return _at(w, name, dev, _F32, (r.heads * r.d if r.norm == 1 else r.d,))


def _first(*ts):
    return next((t for t in ts if t is not None), None)


def veda_qkv_norm_rope(r: veda_rope, q: Optional[torch.Tensor], k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                       wq: Optional[torch.Tensor], wk: Optional[torch.Tensor], q_out: Optional[torch.Tensor],
                       k_out: Optional[torch.Tensor], v_out: Optional[torch.Tensor], stream=None) -> None:
    """Norm of q and k, rotary positions, and token order [B, N, heads, d] (any strides) -> grid order bf16."""
    some = _first(q, k, v)
    if some is None:
        raise ValueError("one of q, k and v is needed")
    dev, dt, n = _device(some, "q, k, v"), some.dtype, r.grid.T * r.grid.H * r.grid.W
    _same_device(r, dev)
    ins, outs = (r.B, n, r.heads, r.d), (r.B, r.heads, n, r.d)
    _call("veda_qkv_norm_rope", dev, stream, ctypes.byref(r), _type(some, "q, k, v"), _tokens(q, r, "q", dev, dt, ins),
          _tokens(k, r, "k", dev, dt, ins), _tokens(v, r, "v", dev, dt, ins), _norm_weight(wq, r, "wq", dev),
          _norm_weight(wk, r, "wk", dev), _at(q_out, "q_out", dev, torch.bfloat16, outs),
          _at(k_out, "k_out", dev, torch.bfloat16, outs), _at(v_out, "v_out", dev, torch.bfloat16, outs))


def _packed_norm_rope(r: veda_rope, qkv: torch.Tensor, wq: Optional[torch.Tensor], wk: Optional[torch.Tensor], outs) -> None:
    """veda_qkv_norm_rope of one packed [B, N, 3, heads, d] tensor of r's sizes into three grid-order tensors that the
    caller has just made: the operands' checks once instead of three times."""
    dev, code, e = _device(qkv, "qkv"), _type(qkv, "qkv"), qkv.element_size()
    sb, sn, s3, sh, sc = qkv.stride()
    if sc != 1:
        raise ValueError("the channels of qkv must be contiguous")
    p, n = qkv.data_ptr(), qkv.shape[1]
    sb, sn, sh = sb if r.B > 1 else 0, sn if n > 1 else 0, sh if r.heads > 1 else 0
    q, k, v = (ctypes.byref(veda_tokens(p + i * s3 * e, sb, sn, sh)) for i in range(3))
    _call("veda_qkv_norm_rope", dev, None, ctypes.byref(r), code, q, k, v, _norm_weight(wq, r, "wq", dev),
          _norm_weight(wk, r, "wk", dev), outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr())


def veda_qkv_norm_rope_backward_workspace(r: veda_rope, device=None) -> int:
    n = _SZ()
    _on_device(device, lambda: _check(LIB.veda_qkv_norm_rope_backward_workspace(ctypes.byref(r), ctypes.byref(n)),
                                      "veda_qkv_norm_rope_backward_workspace"))
    return n.value


def veda_qkv_norm_rope_backward(r: veda_rope, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                                wq: Optional[torch.Tensor], wk: Optional[torch.Tensor], d_q: Optional[torch.Tensor],
                                d_k: Optional[torch.Tensor], d_v: Optional[torch.Tensor], dq: Optional[torch.Tensor],
                                dk: Optional[torch.Tensor], dv: Optional[torch.Tensor], dwq: Optional[torch.Tensor],
                                dwk: Optional[torch.Tensor], workspace: Optional[torch.Tensor], stream=None) -> None:
    """Gradients of veda_qkv_norm_rope for grid-order upstream gradients d_q, d_k, d_v: token-order dq, dk, dv
    (strides of their own) and dwq, dwk.  An operand whose upstream gradient is None is left out."""
    some = _first(dq, dk, dv)
    if some is None:
        raise ValueError("one of dq, dk and dv is needed")
    dev, dt, n, bf = _device(some, "dq, dk, dv"), some.dtype, r.grid.T * r.grid.H * r.grid.W, torch.bfloat16
    _same_device(r, dev)
    ins, outs = (r.B, n, r.heads, r.d), (r.B, r.heads, n, r.d)
    _call("veda_qkv_norm_rope_backward", dev, stream, ctypes.byref(r), _type(some, "dq, dk, dv"),
          _tokens(q, r, "q", dev, dt, ins), _tokens(k, r, "k", dev, dt, ins), _norm_weight(wq, r, "wq", dev),
          _norm_weight(wk, r, "wk", dev), _at(d_q, "d_q", dev, bf, outs), _at(d_k, "d_k", dev, bf, outs),
          _at(d_v, "d_v", dev, bf, outs), _tokens(dq, r, "dq", dev, dt, ins), _tokens(dk, r, "dk", dev, dt, ins),
          _tokens(dv, r, "dv", dev, dt, ins), _norm_weight(dwq, r, "dwq", dev), _norm_weight(dwk, r, "dwk", dev),
          *_scratch(workspace, dev))


def veda_sync_status(stream=None) -> None:
    _check(LIB.veda_sync_status(_stream(stream)), "veda_sync_status")


def veda_set_wait_timeout_ns(ns: int) -> None:
    _check(LIB.veda_set_wait_timeout_ns(int(ns)), "veda_set_wait_timeout_ns")


def veda_selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(LIB.veda_selftest_wait_timeout(int(timeout_ns), _stream(stream)), "veda_selftest_wait_timeout")


def veda_bounds_checked() -> bool:
    """True when the loaded library is the debug build with device-side index checks."""
    return bool(LIB.veda_bounds_checked())


def veda_selftest_bounds(stream=None) -> None:
    """Debug builds: one kernel fails a bounds check on purpose (no memory is
    touched); the next veda_sync_status raises VEDA_ERR_BOUNDS."""
    _check(LIB.veda_selftest_bounds(_stream(stream)), "veda_selftest_bounds")


def veda_version() -> str:
    return LIB.veda_version().decode()
