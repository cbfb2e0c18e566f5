"""Python binding of libsparsp (ctypes): dynamic per-head block-sparse attention
for 3D video-DiT token sequences on one GB300.

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch supplies device memory and the current CUDA stream. There is no CPU
fallback: if the library cannot be loaded, every call raises.

Calls mirror the C ABI in include/sparsp.h (same names, without the prefix).
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# SPARSP_DEBUG=1 in the environment selects the debug build (build(debug=True)),
# whose kernels also bounds-check the addresses they derive themselves
DEBUG = os.environ.get("SPARSP_DEBUG") == "1"
LIB_PATH = os.path.join(_PKG, "libsparsp_debug.so" if DEBUG else "libsparsp.so")

OK, INVALID_ARG, UNSUPPORTED, SHAPE, ALIGN, WORKSPACE, CAPACITY, DATA, CUDA, TIMEOUT = range(10)
F32, BF16 = 0, 1
EST_MEAN, EST_LOWRANK = 0, 1
SCHED_FLAT = 1
KERNEL_PORTABLE = 2
BWD_SPLIT_KV = 4
OUT_RASTER = 8
IN_RASTER = 16
LISTS_SEEN = 32
GRID_CAP_SHIFT = 16
MASKED_SCORE = -1.0e30
NORM_RMS, NORM_HEAD = 1, 2
ROPE_INVERSE, ROPE_IN_BLOCKED, ROPE_OUT_BLOCKED = 1, 2, 4
NORM_ROPE_RMS, NORM_ROPE_BLOCKED = 1, 2
CACHE_CAUSAL = 1


def GRID_CAP(n: int) -> int:
    """Option bits that cap the attention kernels' persistent grid at n CTAs (1..4095)."""
    if not 1 <= n <= 4095:
        raise ValueError("grid cap must be in [1, 4095]")
    return n << GRID_CAP_SHIFT
PROF_SLOTS = 1024


class SparspError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__(f"{call} failed: {status_string(status)} ({status})")


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "T", "Y", "X", "d", "ta", "tb", "tc", "dtype")]

    @property
    def N(self):
        return self.T * self.Y * self.X

    @property
    def Bt(self):
        return self.ta * self.tb * self.tc

    @property
    def nb(self):
        return self.N // self.Bt

    @property
    def rows(self):
        return self.B * self.H * self.nb

    @property
    def torch_dtype(self):
        return torch.float32 if self.dtype == F32 else torch.bfloat16


def make_shape(B, H, T, Y, X, d, ta, tb, tc, dtype) -> Shape:
    if isinstance(dtype, str):
        dtype = F32 if dtype in ("f32", "float32") else BF16
    return Shape(B, H, T, Y, X, d, ta, tb, tc, dtype)


def shape_of(wl) -> Shape:
    """Shape of a workload description with fields B, H, T, Y, X, d, ta, tb, tc, dtype."""
    return make_shape(wl.B, wl.H, wl.T, wl.Y, wl.X, wl.d, wl.ta, wl.tb, wl.tc, wl.dtype)


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SIG = {
    "sparsp_status_string": (ctypes.c_char_p, [_I32]),
    "sparsp_version": (_I32, []),
    "sparsp_device_sm_count": (_I32, []),
    "sparsp_reorder": (_I32, [_P, _P, _P, _I32, _P]),
    "sparsp_block_scores_workspace_size": (ctypes.c_size_t, [_P, _I32, _I32]),
    "sparsp_block_scores": (_I32, [_P, _I32, _P, _P, _P, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "sparsp_reorder_pool": (_I32, [_P, _P, _P, _P, _P]),
    "sparsp_block_scores_pooled_workspace_size": (ctypes.c_size_t, [_P, _I32, _I32]),
    "sparsp_block_scores_pooled": (_I32, [_P, _I32, _P, _P, _P, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "sparsp_select_workspace_size": (ctypes.c_size_t, [_P]),
    "sparsp_select": (_I32, [_P, _P, ctypes.c_float, _I32, _P, _P, _P, ctypes.c_size_t, _P, _P]),
    "sparsp_select_noalloc": (_I32, [_P, _P, ctypes.c_float, _I32, _P, _P, _P, _P]),
    "sparsp_kv_demand": (_I32, [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P, _P,
                                _P]),
    "sparsp_kv_gather": (_I32, [_P, _I32, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P, _P]),
    "sparsp_kv_gather_raster": (_I32, [_P, _I32, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P, _P]),
    "sparsp_placement_workspace_size": (ctypes.c_size_t, [_P]),
    "sparsp_placement": (_I32, [_P, _I32, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]),
    "sparsp_balance_heads": (_I32, [_P, _I32, _I32, _P, _P, _P, _P, _P]),
    "sparsp_augment_workspace_size": (ctypes.c_size_t, [_P, _I32]),
    "sparsp_augment": (_I32, [_P, _I32, _P, _P, _P, _P, _P, _P, ctypes.c_int64, _P, _P, ctypes.c_size_t, _P, _P]),
    "sparsp_predictor_workspace_size": (ctypes.c_size_t, [_P, _I32]),
    "sparsp_predictor_fit": (_I32, [_P, _I32, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "sparsp_lpt_workspace_size": (ctypes.c_size_t, [_P]),
    "sparsp_lpt_schedule": (_I32, [_P, _P, ctypes.c_uint32, _P, _P, ctypes.c_size_t, _P]),
    "sparsp_attn_workspace_size": (ctypes.c_size_t, [_P, _I32]),
    "sparsp_attn_fwd": (_I32, [_P, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, ctypes.c_size_t,
                               ctypes.c_uint32, _P, _P, _P]),
    "sparsp_attn_bwd": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P,
                               ctypes.c_size_t, ctypes.c_uint32, _P, _P, _P]),
    "sparsp_csr_transpose": (_I32, [_P, _P, _P, _P, _P, _P, _P]),
    "sparsp_norm_fwd": (_I32, [_P, ctypes.c_uint32, _P, ctypes.c_int64, _P, _P, ctypes.c_float, _P, _P, _P, _P]),
    "sparsp_norm_workspace_size": (ctypes.c_size_t, [_P, ctypes.c_uint32]),
    "sparsp_norm_bwd": (_I32, [_P, ctypes.c_uint32, _P, _P, ctypes.c_int64, _P, _P, _P, _P, ctypes.c_int64, _P, _P, _P,
                               ctypes.c_size_t, _P]),
    "sparsp_rope_table_size": (ctypes.c_size_t, [_P]),
    "sparsp_rope_table": (_I32, [_P, ctypes.c_double, _P, _P, _P, ctypes.c_size_t, _P]),
    "sparsp_rope": (_I32, [_P, _P, _P, _P, _P, ctypes.c_int64, _P, ctypes.c_int64, ctypes.c_uint32, _P, _P, _P]),
    "sparsp_norm_rope_workspace_size": (ctypes.c_size_t, [_P, _I32]),
    "sparsp_norm_rope_fwd": (_I32, [_P, ctypes.c_uint32, ctypes.c_float, _P, _P, _P, _P, _P, _P, _P]),
    "sparsp_norm_rope_bwd": (_I32, [_P, ctypes.c_uint32, ctypes.c_float, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P,
                                    _P]),
    "sparsp_mask_plan_size": (ctypes.c_size_t, [_P]),
    "sparsp_mask_plan": (_I32, [_P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "sparsp_mask_scores": (_I32, [_P, _P, _P, _P]),
    "sparsp_mask_csr": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P]),
    "sparsp_attn_masked_compacts": (_I32, [_P, _I32]),
    "sparsp_attn_launches": (_I32, [_P, _I32, _I32, ctypes.c_float, ctypes.c_uint32]),
    "sparsp_attn_masked_workspace_size": (ctypes.c_size_t, [_P, _I32]),
    "sparsp_attn_masked_fwd": (_I32, [_P, _P, _P, _P, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _P, _P,
                                      ctypes.c_size_t, ctypes.c_uint32, _P, _P, _P]),
    "sparsp_attn_masked_bwd": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_float, ctypes.c_float, _P, _P, _P,
                                      _P, _P, ctypes.c_size_t, ctypes.c_uint32, _P, _P, _P]),
    "sparsp_cache_extend": (_I32, [_P, _I32, _I32, _P, _P, _P, _I32, _P, _P, _P, _P, _P, ctypes.c_int64, _P, _P, _P]),
    "sparsp_cache_write": (_I32, [_P, _I32, _P, ctypes.c_int64, ctypes.c_int64, _P, ctypes.c_int64, ctypes.c_int64, _P,
                                  ctypes.c_int64, _P, _P, _P, _P, _P, _P]),
    "sparsp_attn_cache_workspace_size": (ctypes.c_size_t, [_P, _I32, _I32, ctypes.c_int64, _I32, _I32]),
    "sparsp_attn_cache_fwd": (_I32, [_P, _I32, _I32, _P, ctypes.c_int64, _P, ctypes.c_int64, _I32, _P, _P, _I32, _P, _P,
                                     _P, _P, _P, _P, ctypes.c_int64, ctypes.c_float, ctypes.c_uint32, _P, _P, _P,
                                     ctypes.c_size_t, _P, _P]),
    "sparsp_diag_umma_tile": (_I32, [_P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "sparsp_diag_wait_timeout": (_I32, [ctypes.c_uint64, _P, _P]),
}


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); run "
                               f"block_sparse_attention_token_gb300.build.build(debug={DEBUG})")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIG.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def status_string(st: int) -> str:
    return lib().sparsp_status_string(int(st)).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None):
    if stream is None:   # the current stream's handle, without a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(name, st):
    if st != OK:
        raise SparspError(name, st)


def _sref(shape: Shape):
    return ctypes.byref(shape)


def _empty(n_bytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(n_bytes), 16), dtype=torch.uint8, device=device)


def _new(stream, dims, dtype, device) -> torch.Tensor:
    """A tensor that a call makes and uses on `stream`: of that stream's memory, so that
    no earlier work on the current stream still uses it, and held for the current
    stream, which reads it afterwards."""
    if stream is None:
        return torch.empty(dims, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(dims, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _refuse(name: str, t, what: str):
    got = (tuple(t.shape), t.dtype, str(t.device), t.stride()) if isinstance(t, torch.Tensor) else t
    raise ValueError(f"{name}: expected {what} on the current CUDA device, got {got}")


def _want(name: str, t, dims, dtype, dev: int, optional: bool = False):
    """Address of a tensor argument of the calls below: contiguous, on device dev
    (the current one), of this shape and dtype. A plain address is passed through."""
    if (t.__class__ is torch.Tensor and t.dtype is dtype and t.shape == dims and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if t is None and optional or isinstance(t, int):
        return t
    if (not isinstance(t, torch.Tensor) or t.shape != dims or t.dtype is not dtype or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(name, t, f"a contiguous {tuple(dims)} {dtype} tensor")
    return t.data_ptr()


def _buffer(name: str, t, dtype, dev: int, optional: bool = False):
    """Address of a buffer of any length: contiguous, on device dev, of this dtype."""
    if t is None and optional or isinstance(t, int):
        return t
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, f"a contiguous {dtype} tensor")
    return t.data_ptr()


def _whole(shape: Shape, name: str, t, optional: bool = False):
    """Refuses a Q-sized tensor of the reorder's layouts that is not one contiguous
    piece of (at least) B*N*H*d values: those calls take its address alone."""
    if t is None and optional or isinstance(t, int):
        return
    s = shape
    n, size = s.B * s.N * s.H * s.d, 4 if s.dtype == F32 else 2
    if not isinstance(t, torch.Tensor) or not t.is_contiguous() or t.numel() < n or t.element_size() != size:
        got = (tuple(t.shape), t.dtype, t.stride()) if isinstance(t, torch.Tensor) else t
        raise ValueError(f"{name}: expected a contiguous tensor of {s.B} x {s.N} x {s.H} x {s.d} {s.torch_dtype} values, "
                         f"got {got}")


def _space(ws, dev: int) -> tuple:
    """(address, bytes) of a workspace tensor."""
    if ws.get_device() != dev or not ws.is_contiguous():
        _refuse("ws", ws, "a contiguous workspace")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _token_stride(shape: Shape, name: str, t, dims, dtype, dev: int) -> tuple:
    """(address, elements between tokens) of a raster tensor [B, N, H, d] that may be
    a slice of a wider one (heads and columns contiguous, batches of N tokens)."""
    if isinstance(t, int):
        return t, 0
    if t is not None and t.shape == dims and t.dtype is dtype and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), 0
        B, N, H, d = dims
        st = t.stride()
        ts = st[1] if N > 1 else st[0] if B > 1 else H * d
        if st[3] == 1 and (H == 1 or st[2] == d) and (B == 1 or st[0] == N * ts) and ts >= H * d:
            return t.data_ptr(), ts
    _refuse(name, t, f"a raster {tuple(dims)} {dtype} tensor with contiguous heads and one stride between tokens")


# ----------------------------------------------------------------- before step 1: token norm, rotary positions

def _norm_flags(rms: bool, per_head: bool) -> int:
    return (NORM_RMS if rms else 0) | (NORM_HEAD if per_head else 0)


def norm_workspace_size(shape: Shape, rms: bool = False, per_head: bool = False) -> int:
    return lib().sparsp_norm_workspace_size(_sref(shape), _norm_flags(rms, per_head))


def norm_fwd(shape: Shape, x, w=None, b=None, eps: float = 1e-6, rms: bool = False, per_head: bool = False, out=None,
             mean=None, rstd=None, stream=None):
    """Layer norm (RMS norm with rms) of raster x [B,N,H,d] over the H*d values of a
    token, or over each head's d values with per_head. x may be a slice of a fused
    projection (one stride between tokens). w, b: float32 [H*d] or [d], or None.
    Returns (y, mean, rstd), the statistics float32 [B,N] ([B,N,H] with per_head);
    mean is None with rms."""
    dims = (shape.B, shape.N, shape.H, shape.d)
    dt, f32, dev = shape.torch_dtype, torch.float32, torch.cuda.current_device()
    px, xs = _token_stride(shape, "x", x, dims, dt, dev)
    cols, stat = ((dims[3],), dims[:3]) if per_head else ((dims[2] * dims[3],), dims[:2])
    if out is None:
        out = _new(stream, dims, dt, x.device)
    if rms:
        mean = None
    elif mean is None:
        mean = _new(stream, stat, f32, x.device)
    if rstd is None:
        rstd = _new(stream, stat, f32, x.device)
    _check("sparsp_norm_fwd", lib().sparsp_norm_fwd(
        _sref(shape), _norm_flags(rms, per_head), px, xs, _want("w", w, cols, f32, dev, True),
        _want("b", b, cols, f32, dev, True), eps, _want("out", out, dims, dt, dev),
        _want("mean", mean, stat, f32, dev, True), _want("rstd", rstd, stat, f32, dev), _stream(stream)))
    return out, mean, rstd


def norm_bwd(shape: Shape, dy, x, w, mean, rstd, rms: bool = False, per_head: bool = False, dx=None, dw=None, db=None,
             ws=None, stream=None):
    """Gradients of norm_fwd from its x, mean (None with rms) and rstd: (dx, dw, db),
    db None with rms unless a buffer is given. dx may be a slice like x."""
    dims = (shape.B, shape.N, shape.H, shape.d)
    dt, f32, dev = shape.torch_dtype, torch.float32, torch.cuda.current_device()
    px, xs = _token_stride(shape, "x", x, dims, dt, dev)
    cols, stat = ((dims[3],), dims[:3]) if per_head else ((dims[2] * dims[3],), dims[:2])
    if dx is None:
        dx = _new(stream, dims, dt, x.device)
    if dw is None:
        dw = _new(stream, cols, f32, x.device)
    if db is None and not rms:
        db = _new(stream, cols, f32, x.device)
    if ws is None:
        ws = _new(stream, max(norm_workspace_size(shape, rms, per_head), 16), torch.uint8, x.device)
    pdx, dxs = _token_stride(shape, "dx", dx, dims, dt, dev)
    _check("sparsp_norm_bwd", lib().sparsp_norm_bwd(
        _sref(shape), _norm_flags(rms, per_head), _want("dy", dy, dims, dt, dev), px, xs,
        _want("w", w, cols, f32, dev, True), None if rms else _want("mean", mean, stat, f32, dev),
        _want("rstd", rstd, stat, f32, dev), pdx, dxs, _want("dw", dw, cols, f32, dev),
        _want("db", db, cols, f32, dev, True), *_space(ws, dev), _stream(stream)))
    return dx, dw, db


class RopeAxes(ctypes.Structure):
    _fields_ = [("cols", _I32 * 3), ("extent", _I32 * 3), ("half", _I32)]


@dataclass
class RopeTable:
    """cos and sin of the three axes (rope_table), kept by the caller."""
    axes: RopeAxes
    table: torch.Tensor


def rope_table(shape: Shape, cols, theta: float = 10000.0, offset=(0.0, 0.0, 0.0), scale=(1.0, 1.0, 1.0),
               extent=None, half: bool = False, stream=None) -> RopeTable:
    """The (cos, sin) table of three-axis rotary positions: cols columns of a head
    turn with the token's frame, row and column; position p of an axis stands for
    offset + scale * p. extent: positions per axis (default: the grid)."""
    cols, ext = [int(c) for c in cols], [int(e) for e in (extent or (shape.T, shape.Y, shape.X))]
    if len(cols) != 3 or len(ext) != 3 or sum(cols) > shape.d or half and sum(cols) != shape.d:
        raise ValueError(f"rope_table: columns {cols} (extent {ext}) do not fit a head of {shape.d} "
                         f"{'paired by halves' if half else ''}")
    axes = RopeAxes((_I32 * 3)(*cols), (_I32 * 3)(*ext), int(half))
    n = lib().sparsp_rope_table_size(ctypes.byref(axes))
    table = _new(stream, max(n // 4, 4), torch.float32, f"cuda:{torch.cuda.current_device()}")
    d3 = ctypes.c_double * 3
    _check("sparsp_rope_table", lib().sparsp_rope_table(
        ctypes.byref(axes), float(theta), ctypes.byref(d3(*offset)), ctypes.byref(d3(*scale)), _ptr(table),
        table.numel() * 4, _stream(stream)))
    return RopeTable(axes, table)


def rope(shape: Shape, table: RopeTable, x, out=None, inverse: bool = False, in_blocked: bool = False,
         out_blocked: bool = True, pos=None, means=None, status=None, stream=None):
    """Turns the rows of x by their positions, from raster [B,N,H,d] (in_blocked:
    blocked [B,H,N,d]) into tile order (out_blocked=False: raster), and returns
    out. inverse: the transposed rotation (gradients). pos: int32 [B,N,3] table
    positions per token, default the grid coordinates. means: float32
    [B,H,nb,d] buffer for the tile means of the turned values. Raster tensors may
    be slices of wider ones (one stride between tokens)."""
    s = shape
    raster, blocked = (s.B, s.N, s.H, s.d), (s.B, s.H, s.N, s.d)
    dt, dev = s.torch_dtype, torch.cuda.current_device()
    if out is None:
        out = _new(stream, blocked if out_blocked else raster, dt, x.device)
    px, xs = ((_want("x", x, blocked, dt, dev), 0) if in_blocked else _token_stride(s, "x", x, raster, dt, dev))
    po, os_ = ((_want("out", out, blocked, dt, dev), 0) if out_blocked
               else _token_stride(s, "out", out, raster, dt, dev))
    flags = ((ROPE_INVERSE if inverse else 0) | (ROPE_IN_BLOCKED if in_blocked else 0)
             | (ROPE_OUT_BLOCKED if out_blocked else 0))
    _check("sparsp_rope", lib().sparsp_rope(
        _sref(s), ctypes.byref(table.axes), _buffer("table", table.table, torch.float32, dev),
        _want("pos", pos, (s.B, s.N, 3), torch.int32, dev, True), px, xs, po, os_, flags,
        _want("means", means, (s.B, s.H, s.nb, s.d), torch.float32, dev, True),
        _buffer("status", status, torch.int32, dev, True), _stream(stream)))
    return out


class NormRope(ctypes.Structure):
    _fields_ = [("heads", _I32), ("x", _P), ("x_stride", ctypes.c_int64), ("dy", _P), ("dy_stride", ctypes.c_int64),
                ("w", _P), ("b", _P), ("out", _P), ("out_stride", ctypes.c_int64), ("means", _P), ("dw", _P), ("db", _P)]


def norm_rope_workspace_size(shape: Shape, heads_k: int = 0) -> int:
    return lib().sparsp_norm_rope_workspace_size(_sref(shape), int(heads_k))


def _head_dims(shape: Shape, name: str, t) -> tuple:
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        _refuse(name, t, "a raster [B, N, heads, d] tensor")
    return shape.B, shape.N, t.shape[2], shape.d


def norm_rope_fwd(shape: Shape, table: RopeTable, q, k=None, q_weight=None, k_weight=None, q_bias=None, k_bias=None,
                  eps: float = 1e-6, rms: bool = False, pos=None, q_out=None, k_out=None, out_blocked: bool = True,
                  q_means=None, k_means=None, status=None, stream=None):
    """norm_fwd(per_head=True) and rope of Q and K in one pass, with one rounding; returns
    (q_out, k_out). q [B,N,H,d] and k [B,N,Hk,d] (or None) are raster and may be slices of a
    fused projection; the results are in tile order, or with out_blocked=False raster,
    and may then be slices too. Weights and biases: float32 [d] or None. Without tile
    order and means the shape's tile does not count (make_shape(1, H, tokens, 1, 1, d, 1, 1,
    1, dtype) with pos for the new tokens of many requests)."""
    s, dt, f32, dev = shape, shape.torch_dtype, torch.float32, torch.cuda.current_device()
    parts, outs = [], []
    for n, x, w, b, out, means in (("q", q, q_weight, q_bias, q_out, q_means), ("k", k, k_weight, k_bias, k_out, k_means)):
        if x is None:
            parts.append(None)
            outs.append(None)
            continue
        raster = _head_dims(s, n, x)
        blocked = (raster[0], raster[2], raster[1], raster[3])
        px, xs = _token_stride(s, n, x, raster, dt, dev)
        if out is None:
            out = _new(stream, blocked if out_blocked else raster, dt, x.device)
        po, os_ = ((_want(n + "_out", out, blocked, dt, dev), 0) if out_blocked
                   else _token_stride(s, n + "_out", out, raster, dt, dev))
        pm = None if means is None else _want(n + "_means", means, (s.B, raster[2], s.nb, s.d), f32, dev)
        parts.append(NormRope(raster[2], px, xs, None, 0, _want(n + "_weight", w, (s.d,), f32, dev, True),
                              _want(n + "_bias", b, (s.d,), f32, dev, True), po, os_, pm, None, None))
        outs.append(out)
    flags = (NORM_ROPE_RMS if rms else 0) | (NORM_ROPE_BLOCKED if out_blocked else 0)
    _check("sparsp_norm_rope_fwd", lib().sparsp_norm_rope_fwd(
        _sref(s), flags, eps, ctypes.byref(table.axes), _buffer("table", table.table, f32, dev),
        _want("pos", pos, (s.B, s.N, 3), torch.int32, dev, True), ctypes.byref(parts[0]),
        None if parts[1] is None else ctypes.byref(parts[1]), _buffer("status", status, torch.int32, dev, True),
        _stream(stream)))
    return outs[0], outs[1]


def norm_rope_bwd(shape: Shape, table: RopeTable, dy_q, dy_k, q, k=None, q_weight=None, k_weight=None,
                  eps: float = 1e-6, rms: bool = False, pos=None, in_blocked: bool = False, dq=None, dk=None, dw=None,
                  db=None, ws=None, status=None, stream=None):
    """Gradients of norm_rope_fwd from its q and k: (dq, dk, [dw of q, of k], [db of q, of k]).
    dy_q, dy_k: gradients of its results, raster (slices too) or with in_blocked in tile
    order. dq and dk are raster and may be slices of one tensor. db is None with rms
    unless buffers are given; entries of k are None without it."""
    s, dt, f32, dev = shape, shape.torch_dtype, torch.float32, torch.cuda.current_device()
    parts, dxs, dws, dbs = [], [], [], []
    for i, (n, x, dy, w, dx) in enumerate((("q", q, dy_q, q_weight, dq), ("k", k, dy_k, k_weight, dk))):
        if x is None:
            for made in (parts, dxs, dws, dbs):
                made.append(None)
            continue
        raster = _head_dims(s, n, x)
        blocked = (raster[0], raster[2], raster[1], raster[3])
        px, xs = _token_stride(s, n, x, raster, dt, dev)
        py, ys = ((_want("dy_" + n, dy, blocked, dt, dev), 0) if in_blocked
                  else _token_stride(s, "dy_" + n, dy, raster, dt, dev))
        if dx is None:
            dx = _new(stream, raster, dt, x.device)
        po, os_ = _token_stride(s, "d" + n, dx, raster, dt, dev)
        gw = _new(stream, (s.d,), f32, x.device) if dw is None or dw[i] is None else dw[i]
        gb = None if db is None else db[i]
        if gb is None and not rms:
            gb = _new(stream, (s.d,), f32, x.device)
        parts.append(NormRope(raster[2], px, xs, py, ys, _want(n + "_weight", w, (s.d,), f32, dev, True), None, po, os_,
                              None, _want("dw", gw, (s.d,), f32, dev), _want("db", gb, (s.d,), f32, dev, True)))
        dxs.append(dx)
        dws.append(gw)
        dbs.append(gb)
    if ws is None:
        heads_k = 0 if k is None else parts[1].heads
        ws = _new(stream, max(norm_rope_workspace_size(s, heads_k), 16), torch.uint8, q.device)
    flags = (NORM_ROPE_RMS if rms else 0) | (NORM_ROPE_BLOCKED if in_blocked else 0)
    _check("sparsp_norm_rope_bwd", lib().sparsp_norm_rope_bwd(
        _sref(s), flags, eps, ctypes.byref(table.axes), _buffer("table", table.table, f32, dev),
        _want("pos", pos, (s.B, s.N, 3), torch.int32, dev, True), ctypes.byref(parts[0]),
        None if parts[1] is None else ctypes.byref(parts[1]), *_space(ws, dev),
        _buffer("status", status, torch.int32, dev, True), _stream(stream)))
    return dxs[0], dxs[1], dws, dbs


# ----------------------------------------------------------------- step 1

def reorder(shape: Shape, x: torch.Tensor, out: torch.Tensor | None = None, inverse: bool = False,
            stream=None) -> torch.Tensor:
    """Raster [B,N,H,d] -> blocked [B,H,N,d] (or back with inverse=True)."""
    _whole(shape, "x", x)
    _whole(shape, "out", out, True)
    if out is None:
        dims = (shape.B, shape.N, shape.H, shape.d) if inverse else (shape.B, shape.H, shape.N, shape.d)
        out = torch.empty(dims, dtype=x.dtype, device=x.device)
    _check("sparsp_reorder", lib().sparsp_reorder(_sref(shape), _ptr(x), _ptr(out), int(inverse), _stream(stream)))
    return out


# ----------------------------------------------------------------- step 2

def block_scores_workspace_size(shape, estimator=EST_MEAN, rank=16) -> int:
    return lib().sparsp_block_scores_workspace_size(_sref(shape), estimator, rank)


def block_scores(shape: Shape, q, k, estimator=EST_MEAN, wq=None, wk=None, rank=16, out=None, ws=None,
                 stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((shape.B, shape.H, shape.nb, shape.nb), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = _empty(block_scores_workspace_size(shape, estimator, rank), q.device)
    _check("sparsp_block_scores", lib().sparsp_block_scores(
        _sref(shape), estimator, _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), rank, _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


def reorder_pool(shape: Shape, x: torch.Tensor, out: torch.Tensor | None = None,
                 means: torch.Tensor | None = None, stream=None):
    """Raster -> blocked, plus the fp32 tile means [B, H, nb, d] from the same pass."""
    _whole(shape, "x", x)
    _whole(shape, "out", out, True)
    if out is None:
        out = torch.empty((shape.B, shape.H, shape.N, shape.d), dtype=x.dtype, device=x.device)
    if means is None:
        means = torch.empty((shape.B, shape.H, shape.nb, shape.d), dtype=torch.float32, device=x.device)
    _check("sparsp_reorder_pool", lib().sparsp_reorder_pool(_sref(shape), _ptr(x), _ptr(out), _ptr(means),
                                                            _stream(stream)))
    return out, means


def pool_means(shape: Shape, x: torch.Tensor, means: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The fp32 tile means [B, H, nb, d] of raster x alone (no reordered copy)."""
    _whole(shape, "x", x)
    if means is None:
        means = torch.empty((shape.B, shape.H, shape.nb, shape.d), dtype=torch.float32, device=x.device)
    _check("sparsp_reorder_pool", lib().sparsp_reorder_pool(_sref(shape), _ptr(x), None, _ptr(means),
                                                            _stream(stream)))
    return means


def block_scores_pooled(shape: Shape, qmeans, kmeans, estimator=EST_MEAN, wq=None, wk=None, rank=16, out=None,
                        ws=None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((shape.B, shape.H, shape.nb, shape.nb), dtype=torch.float32, device=qmeans.device)
    if ws is None:
        n = lib().sparsp_block_scores_pooled_workspace_size(_sref(shape), estimator, rank)
        ws = _empty(n, qmeans.device)
    _check("sparsp_block_scores_pooled", lib().sparsp_block_scores_pooled(
        _sref(shape), estimator, _ptr(qmeans), _ptr(kmeans), _ptr(wq), _ptr(wk), rank, _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out


# ----------------------------------------------------------------- step 3

def select_workspace_size(shape) -> int:
    return lib().sparsp_select_workspace_size(_sref(shape))


def select(shape: Shape, scores, top_p: float, k_floor: int, row_ptr=None, col_idx=None, ws=None,
           status=None, stream=None):
    """Returns (row_ptr, col_idx); col_idx has capacity B*H*nb*nb, nnz = row_ptr[-1]."""
    dev = scores.device
    if row_ptr is None:
        row_ptr = torch.empty(shape.rows + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        col_idx = torch.empty(shape.rows * shape.nb, dtype=torch.int32, device=dev)
    if ws is None:
        ws = _empty(select_workspace_size(shape), dev)
    _check("sparsp_select", lib().sparsp_select(
        _sref(shape), _ptr(scores), float(top_p), int(k_floor), _ptr(row_ptr), _ptr(col_idx), _ptr(ws),
        ws.numel(), _ptr(status), _stream(stream)))
    return row_ptr, col_idx


# ----------------------------------------------------------------- step 4

@dataclass
class DemandOut:
    bitmap: torch.Tensor
    dem_ptr: torch.Tensor
    dem_idx: torch.Tensor
    kg: torch.Tensor | None
    vg: torch.Tensor | None
    bytes: torch.Tensor


def kv_demand(shape: Shape, P: int, row_ptr, col_idx, k=None, v=None, gather_cap: int | None = None,
              out: DemandOut | None = None, status=None, stream=None, owner=None) -> DemandOut:
    """KV demand of P partitions: contiguous query-block ranges, or the block
    owner map `owner` [B, nb] int32 (e.g. from `placement`)."""
    dev = row_ptr.device
    if out is None:
        W = (shape.nb + 31) // 32
        parts = shape.B * shape.H * P
        kg = vg = None
        if k is not None:
            cap = parts * shape.nb if gather_cap is None else gather_cap
            kg = torch.empty((max(cap, 1), shape.Bt, shape.d), dtype=k.dtype, device=dev)
            vg = torch.empty_like(kg)
        out = DemandOut(torch.empty((shape.B, shape.H, P, W), dtype=torch.int32, device=dev),
                        torch.empty(parts + 1, dtype=torch.int32, device=dev),
                        torch.empty(parts * shape.nb, dtype=torch.int32, device=dev), kg, vg,
                        torch.empty(4, dtype=torch.int64, device=dev))
    cap = 0 if out.kg is None else (out.kg.shape[0] if gather_cap is None else gather_cap)
    _check("sparsp_kv_demand", lib().sparsp_kv_demand(
        _sref(shape), int(P), _ptr(row_ptr), _ptr(col_idx), _ptr(owner), _ptr(out.bitmap), _ptr(out.dem_ptr),
        _ptr(out.dem_idx), _ptr(k), _ptr(v), _ptr(out.kg), _ptr(out.vg), int(cap), _ptr(out.bytes),
        _ptr(status), _stream(stream)))
    return out


def kv_gather(shape: Shape, P: int, dem: DemandOut, k, v, gather_cap: int | None = None, status=None,
              stream=None, raster: bool = False) -> DemandOut:
    """The gather of kv_demand alone, into dem.kg / dem.vg, from the lists
    (dem.dem_ptr, dem.dem_idx) of an earlier kv_demand call; it can run on a
    second stream beside attention. raster: k and v in raster order [B, N, H, d]."""
    if dem.kg is None or dem.vg is None:
        raise ValueError("kv_gather needs DemandOut with kg and vg buffers")
    cap = dem.kg.shape[0] if gather_cap is None else gather_cap
    name = "sparsp_kv_gather_raster" if raster else "sparsp_kv_gather"
    _check(name, getattr(lib(), name)(
        _sref(shape), int(P), _ptr(dem.dem_ptr), _ptr(dem.dem_idx), _ptr(k), _ptr(v), _ptr(dem.kg), _ptr(dem.vg),
        int(cap), _ptr(status), _stream(stream)))
    return dem


def placement_workspace_size(shape: Shape) -> int:
    return lib().sparsp_placement_workspace_size(_sref(shape))


def placement(shape: Shape, P: int, row_ptr, col_idx, owner=None, ws=None, status=None,
              stream=None) -> torch.Tensor:
    """Block -> partition assignment [B, nb] int32 from the co-selection
    affinity of the CSR (dependency-aware placement)."""
    dev = row_ptr.device
    if owner is None:
        owner = torch.empty((shape.B, shape.nb), dtype=torch.int32, device=dev)
    if ws is None:
        ws = _empty(placement_workspace_size(shape), dev)
    _check("sparsp_placement", lib().sparsp_placement(
        _sref(shape), int(P), _ptr(row_ptr), _ptr(col_idx), _ptr(owner), _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))
    return owner


@dataclass
class Balance:
    head_rank: torch.Tensor     # int32 [B, H]
    loads: torch.Tensor         # int64 [B, 2, P]: before, after
    migrations: torch.Tensor    # int32 [B]


def balance_heads(shape: Shape, P: int, row_ptr, max_migrations: int, out: Balance | None = None,
                  stream=None) -> Balance:
    """Heads of each batch element on P virtual ranks: contiguous split, then
    greedy migrations of heavy heads off the critical rank."""
    dev = row_ptr.device
    if out is None:
        out = Balance(torch.empty((shape.B, shape.H), dtype=torch.int32, device=dev),
                      torch.empty((shape.B, 2, P), dtype=torch.int64, device=dev),
                      torch.empty(max(shape.B, 4), dtype=torch.int32, device=dev))
    _check("sparsp_balance_heads", lib().sparsp_balance_heads(
        _sref(shape), int(P), int(max_migrations), _ptr(row_ptr), _ptr(out.head_rank), _ptr(out.loads),
        _ptr(out.migrations), _stream(stream)))
    return out


def augment_workspace_size(shape: Shape, P: int) -> int:
    return lib().sparsp_augment_workspace_size(_sref(shape), int(P))


def augment(shape: Shape, P: int, scores, row_ptr, col_idx, head_rank, row_ptr_out=None, col_idx_out=None,
            added=None, ws=None, status=None, stream=None):
    """Slack-aware augmentation of the CSR: each rank's slack up to the critical
    load is filled with its heads' best unselected blocks. Returns
    (row_ptr_out, col_idx_out, added [B, P])."""
    dev = row_ptr.device
    if row_ptr_out is None:
        row_ptr_out = torch.empty(shape.rows + 1, dtype=torch.int32, device=dev)
    if col_idx_out is None:
        col_idx_out = torch.empty(shape.rows * shape.nb, dtype=torch.int32, device=dev)
    if added is None:
        added = torch.empty((shape.B, P), dtype=torch.int64, device=dev)
    if ws is None:
        ws = _empty(augment_workspace_size(shape, P), dev)
    _check("sparsp_augment", lib().sparsp_augment(
        _sref(shape), int(P), _ptr(scores), _ptr(row_ptr), _ptr(col_idx), _ptr(head_rank), _ptr(row_ptr_out),
        _ptr(col_idx_out), int(col_idx_out.numel()), _ptr(added), _ptr(ws), ws.numel(), _ptr(status),
        _stream(stream)))
    return row_ptr_out, col_idx_out, added


def predictor_fit(shape: Shape, qmeans, kmeans, wq, wk, lr: float = 0.0, rank: int | None = None,
                  loss=None, gwq=None, gwk=None, ws=None, stream=None):
    """Loss and gradients of the low-rank predictor against the real block
    scores (mean squared error per head), and the step W -= lr * grad in place
    when lr != 0. Returns (loss [H], gwq, gwk) at the weights before the step."""
    dev = qmeans.device
    rank = wq.shape[-1] if rank is None else rank
    if loss is None:
        loss = torch.empty(shape.H, dtype=torch.float32, device=dev)
    if gwq is None:
        gwq = torch.empty_like(wq)
    if gwk is None:
        gwk = torch.empty_like(wk)
    if ws is None:
        ws = _empty(lib().sparsp_predictor_workspace_size(_sref(shape), int(rank)), dev)
    _check("sparsp_predictor_fit", lib().sparsp_predictor_fit(
        _sref(shape), int(rank), _ptr(qmeans), _ptr(kmeans), _ptr(wq), _ptr(wk), float(lr), _ptr(loss),
        _ptr(gwq), _ptr(gwk), _ptr(ws), ws.numel(), _stream(stream)))
    return loss, gwq, gwk


# ----------------------------------------------------------------- step 5

def lpt_schedule(shape: Shape, row_ptr, flags=0, items=None, stream=None) -> torch.Tensor:
    dev = row_ptr.device
    if items is None:
        items = torch.empty(shape.rows, dtype=torch.int32, device=dev)
    ws = _empty(lib().sparsp_lpt_workspace_size(_sref(shape)), dev)
    _check("sparsp_lpt_schedule", lib().sparsp_lpt_schedule(
        _sref(shape), _ptr(row_ptr), int(flags), _ptr(items), _ptr(ws), ws.numel(), _stream(stream)))
    return items


def csr_transpose(shape: Shape, row_ptr, col_idx, nnz_cap=None, status=None, stream=None):
    dev = row_ptr.device
    col_ptr = torch.empty(shape.rows + 1, dtype=torch.int32, device=dev)
    cap = col_idx.numel() if nnz_cap is None else nnz_cap
    row_idx = torch.empty(max(cap, 4), dtype=torch.int32, device=dev)
    _check("sparsp_csr_transpose", lib().sparsp_csr_transpose(
        _sref(shape), _ptr(row_ptr), _ptr(col_idx), _ptr(col_ptr), _ptr(row_idx), _ptr(status),
        _stream(stream)))
    return col_ptr, row_idx


def attn_launches(shape: Shape, backward: bool = False, plan: bool = False, cap: float = 0.0, flags: int = 0) -> int:
    """The number of kernels that attention with these arguments launches."""
    return lib().sparsp_attn_launches(_sref(shape), int(backward), int(plan), cap, int(flags))


def attn_workspace_size(shape: Shape, backward: bool = False) -> int:
    return lib().sparsp_attn_workspace_size(_sref(shape), int(backward))


def attn_fwd(shape: Shape, q, k, v, row_ptr, col_idx, scale: float = 0.0, o=None, lse=None, ws=None,
             flags: int = 0, prof=None, status=None, stream=None):
    """Returns (O blocked [B,H,N,d], or raster [B,N,H,d] with OUT_RASTER; LSE [B,H,N] fp32)."""
    dev = q.device
    if o is None:
        o = torch.empty((shape.B, shape.N, shape.H, shape.d) if flags & OUT_RASTER else
                        (shape.B, shape.H, shape.N, shape.d), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((shape.B, shape.H, shape.N), dtype=torch.float32, device=dev)
    if ws is None:
        ws = _empty(attn_workspace_size(shape, False), dev)
    _check("sparsp_attn_fwd", lib().sparsp_attn_fwd(
        _sref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr), _ptr(col_idx), float(scale), _ptr(o),
        _ptr(lse), _ptr(ws), ws.numel(), int(flags), _ptr(prof), _ptr(status), _stream(stream)))
    return o, lse


def attn_bwd(shape: Shape, q, k, v, o, lse, dout, row_ptr, col_idx, scale: float = 0.0, dq=None, dk=None,
             dv=None, ws=None, flags: int = 0, prof=None, status=None, stream=None):
    """Returns (dQ, dK, dV), blocked [B,H,N,d] bf16; raster [B,N,H,d] with OUT_RASTER
    in flags (o is then the raster O of attn_fwd with OUT_RASTER)."""
    dev = q.device
    dims = (shape.B, shape.N, shape.H, shape.d) if flags & OUT_RASTER else tuple(q.shape)
    dq = torch.empty(dims, dtype=q.dtype, device=dev) if dq is None else dq
    dk = torch.empty(dims, dtype=k.dtype, device=dev) if dk is None else dk
    dv = torch.empty(dims, dtype=v.dtype, device=dev) if dv is None else dv
    if ws is None:
        ws = _empty(attn_workspace_size(shape, True), dev)
    _check("sparsp_attn_bwd", lib().sparsp_attn_bwd(
        _sref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(row_ptr),
        _ptr(col_idx), float(scale), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(), int(flags),
        _ptr(prof), _ptr(status), _stream(stream)))
    return dq, dk, dv


@dataclass
class MaskPlan:
    """A token mask in tile order with its block ranges (mask_plan), for one shape."""
    dims: tuple
    plan: torch.Tensor


def _mask_dims(s: Shape) -> tuple:
    return s.B, s.T, s.Y, s.X, s.ta, s.tb, s.tc


def mask_plan(shape: Shape, pos, lo, hi, plan: MaskPlan | None = None, stream=None) -> MaskPlan:
    """The token mask in which query n sees key m where lo[n] <= pos[m] < hi[n]
    (int32 [B,N], raster order): documents with pos = lo = number and hi = lo + 1,
    padding with pos = -1 and lo = hi = 0, frames with pos = frame and
    hi = max(frame + 1, prefix). It serves every layer and step with that mask."""
    s, dev = shape, torch.cuda.current_device()
    pos_, lo_, hi_ = (_want(name, t, (s.B, s.N), torch.int32, dev) for name, t in
                      (("pos", pos), ("lo", lo), ("hi", hi)))
    if plan is None:
        plan = MaskPlan(_mask_dims(s), _new(stream, max(lib().sparsp_mask_plan_size(_sref(s)), 16), torch.uint8,
                                            pos.device))
    elif plan.dims != _mask_dims(s):
        raise ValueError(f"mask_plan: the plan is of shape {plan.dims}, not {_mask_dims(s)}")
    _check("sparsp_mask_plan", lib().sparsp_mask_plan(_sref(s), pos_, lo_, hi_, *_space(plan.plan, dev),
                                                      _stream(stream)))
    return plan


def document_mask(shape: Shape, ids):
    """(pos, lo, hi) of mask_plan for documents packed into one grid: ids int32
    [B, N], raster order; a token sees the tokens of its own number, and a token of a
    negative number (padding) sees and is seen by nothing. Numbers are below 2^31 - 1."""
    live = ids >= 0
    pos = torch.where(live, ids, -1).int()
    return pos, torch.where(live, ids, 0).int(), torch.where(live, ids + 1, 0).int()


def frame_mask(shape: Shape, prefix: int = 0, window: int | None = None, device="cuda"):
    """(pos, lo, hi) of mask_plan for generation frame by frame: a token sees its own
    frame and those before it (the last `window` frames of them, its own included),
    and with no window also the first `prefix` frames."""
    if window is not None and (prefix or window < 1):
        raise ValueError("frame_mask: a window is at least one frame and takes no prefix")
    t = (torch.arange(shape.N, device=device) // (shape.Y * shape.X)).expand(shape.B, shape.N)
    lo = torch.zeros_like(t) if window is None else (t - window + 1).clamp(min=0)
    return t.int().contiguous(), lo.int().contiguous(), (t + 1).clamp(min=prefix).int().contiguous()


def _plan_ptr(shape: Shape, mask: MaskPlan | None, dev: int | None = None):
    if mask is None:
        return None
    if mask.dims != _mask_dims(shape):
        raise ValueError(f"the mask plan is of (B, T, Y, X, ta, tb, tc) {mask.dims}, not {_mask_dims(shape)}")
    return mask.plan.data_ptr() if dev is None else _buffer("mask", mask.plan, torch.uint8, dev)


def mask_scores(shape: Shape, mask: MaskPlan, scores, stream=None) -> torch.Tensor:
    """scores [B,H,nb,nb] in place: MASKED_SCORE for block pairs that see nothing of each other."""
    dev = torch.cuda.current_device()
    at = _want("scores", scores, (shape.B, shape.H, shape.nb, shape.nb), torch.float32, dev)
    _check("sparsp_mask_scores", lib().sparsp_mask_scores(_sref(shape), _plan_ptr(shape, mask, dev), at,
                                                          _stream(stream)))
    return scores


def mask_csr(shape: Shape, mask: MaskPlan, row_ptr, col_idx, row_ptr_out=None, col_idx_out=None, status=None,
             stream=None):
    """The rows of a CSR without the block pairs that see nothing of each other (what the
    selection picks of them has no part in attention, and none in its demand or cost).
    Returns (row_ptr_out, col_idx_out); col_idx_out holds at least B*H*nb*nb entries."""
    s, i32, dev = shape, torch.int32, torch.cuda.current_device()
    if row_ptr_out is None:
        row_ptr_out = _new(stream, s.rows + 1, i32, row_ptr.device)
    if col_idx_out is None:
        col_idx_out = _new(stream, s.rows * s.nb, i32, row_ptr.device)
    elif isinstance(col_idx_out, torch.Tensor) and col_idx_out.numel() < s.rows * s.nb:
        raise ValueError(f"mask_csr: col_idx_out holds {col_idx_out.numel()} of up to {s.rows * s.nb} entries")
    _check("sparsp_mask_csr", lib().sparsp_mask_csr(
        _sref(s), _plan_ptr(s, mask, dev), _want("row_ptr", row_ptr, (s.rows + 1,), i32, dev),
        _buffer("col_idx", col_idx, i32, dev), _want("row_ptr_out", row_ptr_out, (s.rows + 1,), i32, dev),
        _buffer("col_idx_out", col_idx_out, i32, dev), _buffer("status", status, i32, dev, True), _stream(stream)))
    return row_ptr_out, col_idx_out


def attn_masked_compacts(shape: Shape, backward: bool = False) -> bool:
    """Does masked attention of this shape run mask_csr on its lists itself (without LISTS_SEEN)?"""
    return lib().sparsp_attn_masked_compacts(_sref(shape), int(backward)) != 0


def attn_masked_workspace_size(shape: Shape, backward: bool = False) -> int:
    return lib().sparsp_attn_masked_workspace_size(_sref(shape), int(backward))


def attn_masked_fwd(shape: Shape, q, k, v, row_ptr, col_idx, scale: float = 0.0, cap: float = 0.0,
                    mask: MaskPlan | None = None, o=None, lse=None, ws=None, flags: int = 0, prof=None, status=None,
                    stream=None):
    """attn_fwd over the keys a token mask lets each query see, with the scores
    capped to cap * tanh(score / cap) when cap > 0. Returns (O, LSE); a query
    that sees nothing has O = 0, LSE = -inf."""
    B, N, H, d = shape.B, shape.N, shape.H, shape.d
    raster, blocked, dt, dev = (B, N, H, d), (B, H, N, d), shape.torch_dtype, torch.cuda.current_device()
    ind, outd = raster if flags & IN_RASTER else blocked, raster if flags & OUT_RASTER else blocked
    if o is None:
        o = _new(stream, outd, dt, q.device)
    if lse is None:
        lse = _new(stream, (B, H, N), torch.float32, q.device)
    if ws is None:
        ws = _new(stream, max(attn_masked_workspace_size(shape, False), 16), torch.uint8, q.device)
    _check("sparsp_attn_masked_fwd", lib().sparsp_attn_masked_fwd(
        _sref(shape), _want("q", q, ind, dt, dev), _want("k", k, ind, dt, dev), _want("v", v, ind, dt, dev),
        _want("row_ptr", row_ptr, (shape.rows + 1,), torch.int32, dev), _buffer("col_idx", col_idx, torch.int32, dev),
        scale, cap, _plan_ptr(shape, mask, dev), _want("o", o, outd, dt, dev),
        _want("lse", lse, (B, H, N), torch.float32, dev),
        *_space(ws, dev), int(flags), _buffer("prof", prof, torch.int64, dev, True),
        _buffer("status", status, torch.int32, dev, True), _stream(stream)))
    return o, lse


def attn_masked_bwd(shape: Shape, q, k, v, o, lse, dout, row_ptr, col_idx, scale: float = 0.0, cap: float = 0.0,
                    mask: MaskPlan | None = None, dq=None, dk=None, dv=None, ws=None, flags: int = 0, prof=None,
                    status=None, stream=None):
    """Gradients of attn_masked_fwd, (dQ, dK, dV); layouts as attn_bwd."""
    B, N, H, d = shape.B, shape.N, shape.H, shape.d
    raster, blocked, dt, dev = (B, N, H, d), (B, H, N, d), shape.torch_dtype, torch.cuda.current_device()
    outd = raster if flags & OUT_RASTER else blocked
    dq, dk, dv = (_new(stream, outd, dt, q.device) if t is None else t for t in (dq, dk, dv))
    if ws is None:
        ws = _new(stream, max(attn_masked_workspace_size(shape, True), 16), torch.uint8, q.device)
    _check("sparsp_attn_masked_bwd", lib().sparsp_attn_masked_bwd(
        _sref(shape), _want("q", q, blocked, dt, dev), _want("k", k, blocked, dt, dev),
        _want("v", v, blocked, dt, dev), _want("o", o, outd, dt, dev),
        _want("lse", lse, (B, H, N), torch.float32, dev), _want("dout", dout, blocked, dt, dev),
        _want("row_ptr", row_ptr, (shape.rows + 1,), torch.int32, dev), _buffer("col_idx", col_idx, torch.int32, dev),
        scale, cap, _plan_ptr(shape, mask, dev), _want("dq", dq, outd, dt, dev), _want("dk", dk, outd, dt, dev),
        _want("dv", dv, outd, dt, dev), *_space(ws, dev), int(flags),
        _buffer("prof", prof, torch.int64, dev, True), _buffer("status", status, torch.int32, dev, True),
        _stream(stream)))
    return dq, dk, dv


def diag_umma_tile(a: torch.Tensor, b: torch.Tensor, mode: int, lbo: int = 16384, sbo: int = 1024,
                   status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One 128x128x128 bf16 tcgen05 tile product (layout diagnostic, include/sparsp_diag.h).
    status: device int32 word that receives SPARSP_ERR_TIMEOUT if a bounded wait
    expires (a fresh zeroed one is used when None; check it after synchronising)."""
    d = torch.empty((128, 128), dtype=torch.float32, device=a.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=a.device)
    _check("sparsp_diag_umma_tile", lib().sparsp_diag_umma_tile(_ptr(a), _ptr(b), _ptr(d), int(mode), int(lbo),
                                                                int(sbo), _ptr(status), _stream(stream)))
    return d


def diag_wait_timeout(limit_ns: int, status: torch.Tensor, stream=None) -> None:
    """Runs the tensor-core kernels' bounded wait on a barrier nothing completes
    (include/sparsp_diag.h); *status receives SPARSP_ERR_TIMEOUT after limit_ns."""
    _check("sparsp_diag_wait_timeout", lib().sparsp_diag_wait_timeout(int(limit_ns), _ptr(status), _stream(stream)))


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


from .cache import (CachePool, CacheShape, attn_cache_fwd, attn_cache_workspace_size, block_pool,  # noqa: E402,F401
                    cache_extend, cache_write)
from .pipeline import GraphedStep, Pipeline, QKNorm  # noqa: E402,F401
from .streaming import HostPipeline  # noqa: E402,F401
