"""Python binding of libmxg.so (include/mxg.h): argument marshalling only.

Every function here has the name of the C entry point it calls and passes
device pointers and sizes straight through; all arithmetic runs in the
library's sm_103a kernels.  torch tensors are used as device buffers and the
current torch stream is the default stream.  There is no fallback: if the
library is missing or the call fails, an exception is raised.

The ``alloc_*`` helpers only size and allocate output buffers (torch.empty)
for the shapes include/mxg.h documents.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxg.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "mxg.h")

# enums of include/mxg.h
MXG_OK = 0
MXG_MXFP8_E4M3, MXG_NVFP4_ROWSCALED = 1, 2
MXG_ROWWISE, MXG_COLWISE, MXG_BOTH = 1, 2, 3
MXG_FPROP_TN, MXG_WGRAD_NT, MXG_DGRAD_NN = 0, 1, 2
MXG_OUT_F32, MXG_OUT_BF16 = 0, 1
MXG_F32, MXG_BF16, MXG_F16 = 0, 1, 2
MXG_GATE_NONE, MXG_GATE_ROW, MXG_GATE_COL, MXG_GATE_FULL = 0, 1, 2, 3
MXG_SCORE_SOFTMAX, MXG_SCORE_SIGMOID = 0, 1
MXG_ACT_SILU, MXG_ACT_GELU_TANH = 0, 1
MXG_DEV_NEG_SIZE, MXG_DEV_MISALIGNED, MXG_DEV_SUM_OVER_CAPACITY = 1, 2, 4
MXG_DEV_BOUNDS, MXG_DEV_TIMEOUT = 8, 16
STATUS_NAMES = {0: "MXG_OK", 1: "MXG_ERR_INVALID_ARG", 2: "MXG_ERR_ALIGNMENT",
                3: "MXG_ERR_UNSUPPORTED_ARCH", 4: "MXG_ERR_LAUNCH",
                5: "MXG_ERR_WORKSPACE_TOO_SMALL", 6: "MXG_ERR_UNSUPPORTED"}


class MxgError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__("%s failed: %s (%d)" % (fn, STATUS_NAMES.get(code, "?"), code))
        self.code = code


class Operand(ctypes.Structure):
    """mxg_operand_t"""
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("outer", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64)]


class BlockNorm(ctypes.Structure):
    """mxg_block_norm_t"""
    _fields_ = [("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("w_post", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("gate_mode", ctypes.c_int),
                ("res_scale", ctypes.c_float), ("x_out", ctypes.c_void_p),
                ("ldxo", ctypes.c_int64), ("w_pre", ctypes.c_void_p), ("n_out", ctypes.c_void_p),
                ("ldn", ctypes.c_int64), ("eps", ctypes.c_float)]


class BlockNormGrad(ctypes.Structure):
    """mxg_block_norm_grad_t"""
    _fields_ = [("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("w_post", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("gate_mode", ctypes.c_int),
                ("res_scale", ctypes.c_float), ("w_pre", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("dx_out", ctypes.c_void_p), ("lddxo", ctypes.c_int64),
                ("dn", ctypes.c_void_p), ("lddn", ctypes.c_int64), ("dx", ctypes.c_void_p),
                ("lddx", ctypes.c_int64), ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
                ("dw_post", ctypes.c_void_p), ("dw_pre", ctypes.c_void_p),
                ("dgate", ctypes.c_void_p), ("lddg", ctypes.c_int64)]


class Grad(ctypes.Structure):
    """mxg_grad_t"""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_type", ctypes.c_int), ("dst_type", ctypes.c_int)]


class Route(ctypes.Structure):
    """mxg_route_t"""
    _fields_ = [("dtype", ctypes.c_int), ("tokens", ctypes.c_int64), ("experts", ctypes.c_int32),
                ("k", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("score", ctypes.c_int), ("normalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("balance", ctypes.c_float),
                ("expert", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("loss", ctypes.c_void_p), ("slope", ctypes.c_void_p),
                ("row_of", ctypes.c_void_p), ("group_ws", ctypes.c_void_p),
                ("align", ctypes.c_int32), ("rows_capacity", ctypes.c_int64),
                ("last_dim", ctypes.c_int64)]


class RouteGrad(ctypes.Structure):
    """mxg_route_grad_t"""
    _fields_ = [("dtype", ctypes.c_int), ("tokens", ctypes.c_int64), ("experts", ctypes.c_int32),
                ("k", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("expert", ctypes.c_void_p), ("score", ctypes.c_int), ("normalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dweight", ctypes.c_void_p),
                ("slope", ctypes.c_void_p), ("dloss", ctypes.c_void_p),
                ("dlogits", ctypes.c_void_p), ("ldd", ctypes.c_int64)]


class ExpertRows(ctypes.Structure):
    """mxg_expert_rows_t"""
    _fields_ = [("dtype", ctypes.c_int), ("n", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("k", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("rows_capacity", ctypes.c_int64), ("tokens", ctypes.c_void_p),
                ("ldt", ctypes.c_int64), ("rows", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("row_of", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("y_rows", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("dweight", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("group_ws", ctypes.c_void_p)]


class GatedAct(ctypes.Structure):
    """mxg_gated_act_t"""
    _fields_ = [("dtype", ctypes.c_int), ("act", ctypes.c_int), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("gated", ctypes.c_int32), ("G", ctypes.c_int32),
                ("group_ws", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64),
                ("up", ctypes.c_void_p), ("ldu", ctypes.c_int64), ("h", ctypes.c_void_p),
                ("ldh", ctypes.c_int64), ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64),
                ("sf", ctypes.c_void_p), ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64),
                ("dgate", ctypes.c_void_p), ("lddg", ctypes.c_int64), ("dup", ctypes.c_void_p),
                ("lddu", ctypes.c_int64)]


def _operand(T, elems_per_byte: int) -> Operand:
    """(data, scale[, outer]) -> mxg_operand_t.  A 2-D data tensor passes its
    leading dimension (row stride in elements), so a view of rows inside a
    wider buffer is described as such; rows and cols are left to the library
    (0: as the GEMM mode implies)."""
    data = T[0]
    ld = 0
    if isinstance(data, torch.Tensor) and data.dim() == 2:
        ld = data.stride(0) * elems_per_byte
    return Operand(_p(data), _p(T[1]), _p(T[2]) if len(T) > 2 else None, 0, 0, ld)


_lib = None


def load() -> ctypes.CDLL:
    """Load libmxg.so (built by moe_grouped_block_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmxg.so is not built: run `python -m moe_grouped_block_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, c_int, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int,
                                   ctypes.c_size_t)
        L.mxg_offsets_workspace_bytes.restype = sz
        L.mxg_offsets_workspace_bytes.argtypes = [c_int]
        L.mxg_group_offsets.restype = c_int
        L.mxg_group_offsets.argtypes = [vp, c_int, c_int, i64, i64, i64, vp, vp, vp]
        L.mxg_group_quantize.restype = c_int
        L.mxg_group_quantize.argtypes = [c_int, c_int, vp, i64, i64, vp, c_int, vp, vp, vp, vp, vp,
                                         vp, vp, vp]
        L.mxg_grouped_gemm.restype = c_int
        L.mxg_grouped_gemm.argtypes = [c_int, c_int, ctypes.POINTER(Operand), ctypes.POINTER(Operand),
                                       vp, c_int, i64, i64, i64, vp, vp, vp, vp, c_int, vp, sz, vp,
                                       vp]
        L.mxg_grouped_gemm_debug.restype = c_int
        L.mxg_grouped_gemm_debug.argtypes = [c_int, c_int, ctypes.POINTER(Operand),
                                             ctypes.POINTER(Operand), vp, c_int, i64, i64, i64, vp,
                                             vp, vp, vp, c_int, vp, c_int, c_int, c_int, i64, vp]
        L.mxg_grouped_gemm_workspace_bytes.restype = sz
        L.mxg_grouped_gemm_workspace_bytes.argtypes = [c_int, c_int, c_int, i64, i64]
        L.mxg_dequantize.restype = c_int
        L.mxg_dequantize.argtypes = [c_int, c_int, vp, vp, vp, i64, i64, vp, c_int, vp]
        L.mxg_status_string.restype = ctypes.c_char_p
        L.mxg_status_string.argtypes = [c_int]
        L.mxg_version.restype = c_int
        L.mxg_version.argtypes = []
        L.mxg_launch_count.restype = ctypes.c_uint64
        L.mxg_launch_count.argtypes = []
        L.mxg_unaligned_rows_capacity.restype = i64
        L.mxg_unaligned_rows_capacity.argtypes = [i64, c_int]
        L.mxg_group_offsets_unaligned.restype = c_int
        L.mxg_group_offsets_unaligned.argtypes = [vp, c_int, c_int, i64, i64, i64, vp, vp, vp]
        L.mxg_group_quantize_unaligned.restype = c_int
        L.mxg_group_quantize_unaligned.argtypes = [c_int, vp, i64, i64, vp, c_int, vp, vp, vp, vp,
                                                   vp, vp]
        L.mxg_grouped_gemm_unaligned.restype = c_int
        L.mxg_grouped_gemm_unaligned.argtypes = [c_int, ctypes.POINTER(Operand),
                                                 ctypes.POINTER(Operand), vp, c_int, i64, i64, i64,
                                                 vp, vp, vp, vp, c_int, vp, vp]
        L.mxg_grouped_gemm_16bit.restype = c_int
        L.mxg_grouped_gemm_16bit.argtypes = [c_int, c_int, vp, i64, vp, i64, vp, c_int, i64, i64,
                                             i64, vp, vp, vp, i64, c_int, vp, vp]
        L.mxg_block_norm.restype = c_int
        L.mxg_block_norm.argtypes = [ctypes.POINTER(BlockNorm), vp]
        L.mxg_block_norm_workspace_bytes.restype = sz
        L.mxg_block_norm_workspace_bytes.argtypes = [i64, i64]
        L.mxg_block_norm_backward.restype = c_int
        L.mxg_block_norm_backward.argtypes = [ctypes.POINTER(BlockNormGrad), vp, sz, vp]
        L.mxg_grad_workspace_bytes.restype = sz
        L.mxg_grad_workspace_bytes.argtypes = []
        L.mxg_grad_norm.restype = c_int
        L.mxg_grad_norm.argtypes = [vp, c_int, vp, vp, sz, vp]
        L.mxg_grad_clip.restype = c_int
        L.mxg_grad_clip.argtypes = [vp, c_int, ctypes.c_float, vp, vp, sz, vp]
        L.mxg_route_workspace_bytes.restype = sz
        L.mxg_route_workspace_bytes.argtypes = [i64, c_int, c_int]
        L.mxg_route.restype = c_int
        L.mxg_route.argtypes = [vp, vp, sz, vp, vp]
        L.mxg_route_rows.restype = c_int
        L.mxg_route_rows.argtypes = [vp, i64, c_int, c_int, c_int, i64, i64, vp, vp, vp, vp, sz, vp,
                                     vp]
        L.mxg_route_backward.restype = c_int
        L.mxg_route_backward.argtypes = [vp, vp]
        for f in (L.mxg_dispatch, L.mxg_combine, L.mxg_combine_backward):
            f.restype = c_int
            f.argtypes = [vp, vp]
        for f in (L.mxg_gated_act, L.mxg_gated_act_backward):
            f.restype = c_int
            f.argtypes = [vp, vp]
        _lib = L
    return _lib


def declared_functions() -> list:
    """Names of the functions include/mxg.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(mxg_[a-z0-9_]+)\s*\(", text)))


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libmxg takes device tensors; got a %s tensor" % t.device)
    return t.data_ptr()


def _word(t) -> int | None:
    """A status word: kernels write four bytes on a boundary of four."""
    if isinstance(t, torch.Tensor) and (t.itemsize < 4 or t.numel() < 1):
        raise ValueError("dev_status: expected an int32 word: got %s of %s"
                         % (tuple(t.shape), t.dtype))
    return _p(t)


def _dense(workspace):
    """A workspace whose bytes are those from its address on."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("a workspace must be contiguous: got strides %s" % (workspace.stride(),))
    return workspace


# the handle alone of the current stream of a device: making the Stream object
# costs 6 us, as much as the rest of a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, code: int) -> None:
    if code != MXG_OK:
        raise MxgError(fn, code)


# ----------------------------------------------------------------- entry points
def mxg_offsets_workspace_bytes(G: int) -> int:
    return load().mxg_offsets_workspace_bytes(G)


def mxg_group_offsets(sizes: torch.Tensor, multiplier: int, last_dim: int, rows_capacity: int,
                      ws: torch.Tensor, dev_status: torch.Tensor | None = None, stream=None) -> None:
    assert sizes.dtype in (torch.int32, torch.int64) and ws.dtype == torch.int64
    _check("mxg_group_offsets",
           load().mxg_group_offsets(_p(sizes), 1 if sizes.dtype == torch.int64 else 0, sizes.numel(),
                                    multiplier, last_dim, rows_capacity, _p(ws), _word(dev_status),
                                    _s(stream)))


def mxg_group_quantize(fmt: int, layout: int, x: torch.Tensor, rows_capacity: int, cols: int,
                       group_ws: torch.Tensor | None, G: int, q_row=None, sf_row=None, q_col=None,
                       sf_col=None, outer_row=None, dev_status=None, stream=None,
                       outer_col=None) -> None:
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    _check("mxg_group_quantize",
           load().mxg_group_quantize(fmt, layout, _p(x), rows_capacity, cols, _p(group_ws), G,
                                     _p(q_row), _p(sf_row), _p(q_col), _p(sf_col), _p(outer_row),
                                     _p(outer_col), _word(dev_status), _s(stream)))


def mxg_grouped_gemm(fmt: int, mode: int, A: tuple, B: tuple, group_ws: torch.Tensor, G: int,
                     M_cap: int, N: int, K: int, alpha=None, beta=None, C=None,
                     out_type: int = MXG_OUT_F32, workspace=None, workspace_bytes: int = 0,
                     dev_status=None, stream=None, bias=None) -> None:
    """A, B: (data, scale, outer-or-None) device tensors."""
    epb = 2 if fmt == MXG_NVFP4_ROWSCALED else 1
    a, b = _operand(A, epb), _operand(B, epb)
    _check("mxg_grouped_gemm",
           load().mxg_grouped_gemm(fmt, mode, ctypes.byref(a), ctypes.byref(b), _p(group_ws), G,
                                   M_cap, N, K, _p(alpha), _p(beta), _p(bias), _p(C), out_type,
                                   _p(workspace),
                                   workspace_bytes, _word(dev_status), _s(stream)))


def mxg_grouped_gemm_debug(fmt: int, mode: int, A: tuple, B: tuple, group_ws, G: int, M_cap: int,
                           N: int, K: int, alpha=None, beta=None, C=None,
                           out_type: int = MXG_OUT_F32, dev_status=None, tile_n: int = 0,
                           stage_bytes: int = 0, inject_flags: int = 0, wait_timeout_ns: int = 0,
                           stream=None, bias=None) -> None:
    epb = 2 if fmt == MXG_NVFP4_ROWSCALED else 1
    a, b = _operand(A, epb), _operand(B, epb)
    _check("mxg_grouped_gemm_debug",
           load().mxg_grouped_gemm_debug(fmt, mode, ctypes.byref(a), ctypes.byref(b), _p(group_ws),
                                         G, M_cap, N, K, _p(alpha), _p(beta), _p(bias), _p(C),
                                         out_type, _word(dev_status), tile_n, stage_bytes,
                                         inject_flags, wait_timeout_ns, _s(stream)))


def mxg_grouped_gemm_workspace_bytes(fmt: int, mode: int, G: int, M_cap: int, N: int) -> int:
    return load().mxg_grouped_gemm_workspace_bytes(fmt, mode, G, M_cap, N)


def mxg_dequantize(fmt: int, layout: int, q, sf, outer, rows: int, cols: int, out,
                   out_type: int = MXG_OUT_F32, stream=None) -> None:
    _check("mxg_dequantize",
           load().mxg_dequantize(fmt, layout, _p(q), _p(sf), _p(outer), rows, cols, _p(out),
                                 out_type, _s(stream)))


def mxg_unaligned_rows_capacity(rows_capacity: int, G: int) -> int:
    return load().mxg_unaligned_rows_capacity(rows_capacity, G)


def mxg_group_offsets_unaligned(sizes: torch.Tensor, multiplier: int, last_dim: int,
                                rows_capacity: int, ws: torch.Tensor,
                                dev_status: torch.Tensor | None = None, stream=None) -> None:
    assert sizes.dtype in (torch.int32, torch.int64) and ws.dtype == torch.int64
    _check("mxg_group_offsets_unaligned",
           load().mxg_group_offsets_unaligned(_p(sizes), 1 if sizes.dtype == torch.int64 else 0,
                                              sizes.numel(), multiplier, last_dim, rows_capacity,
                                              _p(ws), _word(dev_status), _s(stream)))


def mxg_group_quantize_unaligned(layout: int, x: torch.Tensor, rows_capacity: int, cols: int,
                                 group_ws: torch.Tensor, G: int, q_row=None, sf_row=None,
                                 q_col=None, sf_col=None, dev_status=None, stream=None) -> None:
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    _check("mxg_group_quantize_unaligned",
           load().mxg_group_quantize_unaligned(layout, _p(x), rows_capacity, cols, _p(group_ws), G,
                                               _p(q_row), _p(sf_row), _p(q_col), _p(sf_col),
                                               _word(dev_status), _s(stream)))


def mxg_grouped_gemm_unaligned(mode: int, A: tuple, B: tuple, group_ws: torch.Tensor, G: int,
                               M_cap: int, N: int, K: int, alpha=None, beta=None, C=None,
                               out_type: int = MXG_OUT_F32, dev_status=None, stream=None,
                               bias=None) -> None:
    """A, B: (data, scale) device tensors (MXFP8)."""
    a, b = _operand(A[:2], 1), _operand(B[:2], 1)
    _check("mxg_grouped_gemm_unaligned",
           load().mxg_grouped_gemm_unaligned(mode, ctypes.byref(a), ctypes.byref(b), _p(group_ws),
                                             G, M_cap, N, K, _p(alpha), _p(beta), _p(bias), _p(C),
                                             out_type, _word(dev_status), _s(stream)))


# ------------------------------------------------ 16-bit operators of an expert block
_DTYPES = {torch.float32: MXG_F32, torch.bfloat16: MXG_BF16, torch.float16: MXG_F16}


def _ld(t) -> int:
    """Elements between the rows of a matrix whose rows are contiguous; 0 where
    they follow one another."""
    if t is None or t.is_contiguous():
        return 0
    stride = t.stride()
    if len(stride) < 2:
        raise ValueError("a vector must be contiguous")
    rows, cols = t.shape[-2:]
    if stride[-1] != 1 and cols > 1:
        raise ValueError("rows must be contiguous (stride %d between their elements)" % stride[-1])
    # the stride of a dimension of size 1 says nothing
    if rows > 1 and stride[-2] < cols:
        raise ValueError("rows overlap (stride %d, %d elements): a broadcast matrix has to be "
                         "materialised" % (stride[-2], cols))
    return stride[-2] if rows > 1 else max(stride[-2], cols)


def _operand16(t, name: str, want: tuple) -> int:
    """Elements between the rows of the matrix [rows, cols] that t holds, or of the
    experts [G, rows, cols] one after the other, and 0 where they are dense.  t may
    have more rows (or experts), and more columns in a row; a contiguous t counts as
    its reshape."""
    per = want[1] if len(want) == 3 else 0
    rows, cols = want[0] * (per or 1), want[-1]
    if rows < 0 or cols < 1:
        return 0  # the library refuses the sizes
    shape, stride = t.shape, t.stride()
    dense = t.is_contiguous() and _reshapes_to(shape, rows, cols, per)
    if not dense:
        have = shape[0] * shape[1] if len(shape) == 3 else shape[0]
        if (len(shape) not in (2, 3) or shape[-1] < cols or have < rows
                or (len(shape) == 3 and per and shape[1] != per)):
            raise ValueError("%s: expected %s: got %s" % (name, want, tuple(shape)))
        if stride[-1] != 1 and cols > 1:
            raise ValueError("%s: rows must be contiguous (stride %d between their elements)"
                             % (name, stride[-1]))
    if rows <= 1:  # no stride to keep: any multiple of 8 serves
        return (cols + 7) // 8 * 8
    if dense:
        return 0
    one = len(shape) == 3 and shape[1] == 1
    ld = stride[0] if one else stride[-2]
    if ld < cols:
        raise ValueError("%s: rows overlap (stride %d, %d elements)" % (name, ld, cols))
    if len(shape) == 3 and rows > shape[1] and stride[0] != shape[1] * ld:
        raise ValueError("%s: experts must lie one after the other (stride %d, want %d)"
                         % (name, stride[0], shape[1] * ld))
    return ld


def _reshapes_to(shape, rows: int, cols: int, per: int) -> bool:
    """Whether a contiguous tensor of this shape starts with `rows` dense rows: its last
    dimensions together are the columns, or its elements are just as many."""
    n = math.prod(shape)
    if n < rows * cols:
        return False
    if len(shape) == 1:
        return True
    if len(shape) == 3 and per and shape[-1] == cols:
        return shape[1] == per
    width = 1
    for d in reversed(shape):
        width *= d
        if width >= cols:
            break
    return width == cols or (n == rows * cols and shape[-1] % cols == 0)


def _per_group(t, name: str, G: int) -> None:
    """alpha or beta: a contiguous fp32 vector of at least G elements."""
    if not isinstance(t, int) and (t.dtype is not torch.float32 or t.numel() < G
                                   or not t.is_contiguous()):
        raise ValueError("%s: expected %d contiguous fp32 elements: got %s of %s"
                         % (name, G, tuple(t.shape), t.dtype))


def mxg_grouped_gemm_16bit(mode: int, A: torch.Tensor, B: torch.Tensor, group_ws: torch.Tensor,
                           G: int, M_cap: int, N: int, K: int, alpha=None, beta=None,
                           C: torch.Tensor = None, dev_status=None, stream=None) -> None:
    """A, B: bf16 or fp16 device tensors of at least the rows and columns that the mode
    implies ([M_cap, N or K]; weights [G, N, K] or [G*N, K]), of which the first ones
    count; rows may be strided.  C: fp32 or the operands' type."""
    kind, out = _DTYPES.get(A.dtype), _DTYPES.get(C.dtype)
    if not kind or out is None or B.dtype is not A.dtype:  # MXG_F32 is 0
        raise ValueError("operands of one 16-bit type, C of that or fp32: got %s, %s, %s"
                         % (A.dtype, B.dtype, C.dtype))
    assert group_ws.dtype == torch.int64
    if group_ws.numel() < G or not group_ws.is_contiguous():
        raise ValueError("group_ws: expected the workspace of %d groups: got %s"
                         % (G, tuple(group_ws.shape)))
    for v, name in ((alpha, "alpha"), (beta, "beta")):
        if v is not None:
            _per_group(v, name, G)
    a = (M_cap, K if mode == MXG_FPROP_TN else N)
    if mode == MXG_WGRAD_NT:
        b, c = (M_cap, K), (G, N, K)
    else:
        b, c = (G, N, K), (M_cap, N if mode == MXG_FPROP_TN else K)
    # (a dense single row of a width that is no multiple of 8 is given a stride that is)
    if ((not (N | K) & 7 or (M_cap > 1 and N > 1)) and A.shape == a and B.shape == b
            and C.shape == c and A.is_contiguous() and B.is_contiguous() and C.is_contiguous()):
        lda = ldb = ldc = 0  # as nearly all are
    else:
        lda, ldb, ldc = _operand16(A, "A", a), _operand16(B, "B", b), _operand16(C, "C", c)
    _check("mxg_grouped_gemm_16bit",
           load().mxg_grouped_gemm_16bit(kind, mode, _p(A), lda, _p(B), ldb, _p(group_ws), G,
                                         M_cap, N, K, _p(alpha), _p(beta), _p(C), ldc, out,
                                         _word(dev_status), _s(stream)))


def _same_type(tensors) -> int:
    """The mxg_dtype_t of those that are given."""
    kind = None
    for t in tensors:
        if t is not None and t.dtype is not kind:
            if kind is not None:
                raise ValueError("tensors of one type expected: got %s and %s" % (kind, t.dtype))
            kind = t.dtype
    if kind not in _DTYPES:
        raise ValueError("expected fp32, bf16 or fp16: got %s" % kind)
    return _DTYPES[kind]


def _same_shape(x, tensors) -> None:
    shape = x.shape
    for t in tensors:
        if t is not None and t.shape != shape:
            raise ValueError("the [rows, cols] tensors differ in shape: %s and %s"
                             % (tuple(shape), tuple(t.shape)))


def _vector(t, n: int, f32: bool = False) -> None:
    """A contiguous vector of n elements, or none."""
    if t is not None and (t.numel() != n or not t.is_contiguous() or
                          (f32 and t.dtype is not torch.float32)):
        raise ValueError("expected a contiguous vector of %d%s: got %s of %s"
                         % (n, " fp32 elements" if f32 else "", tuple(t.shape), t.dtype))


def _gate(gate, mode: int, x, broadcast_f32: bool) -> None:
    """A gate of the given mode or (broadcast_f32) its gradient."""
    if gate is None:
        return
    if mode == MXG_GATE_ROW:
        _vector(gate, x.shape[0], True)
    elif mode == MXG_GATE_COL:
        _vector(gate, x.shape[1], broadcast_f32)
    elif mode != MXG_GATE_FULL or gate.shape != x.shape:
        raise ValueError("a gate of mode %d does not have the shape %s" % (mode, tuple(gate.shape)))


def mxg_block_norm(x: torch.Tensor, y=None, w_post=None, gate=None, gate_mode: int = MXG_GATE_NONE,
                   res_scale: float = 1.0, x_out=None, w_pre=None, n_out=None, eps: float = 1e-6,
                   stream=None) -> None:
    """x, y, x_out, n_out: [rows, cols] (rows may be strided)."""
    rows, cols = x.shape
    full = gate_mode == MXG_GATE_FULL
    dtype = _same_type((y, n_out, w_post, w_pre, gate if gate_mode >= MXG_GATE_COL else None))
    res = _same_type((x, x_out))
    _same_shape(x, (y, x_out, n_out))
    _vector(w_post, cols)
    _vector(w_pre, cols)
    _gate(gate, gate_mode, x, False)
    d = BlockNorm(dtype, res, rows, cols, _p(x), _ld(x), _p(y), _ld(y), _p(w_post), _p(gate),
                  _ld(gate) if full else 0, gate_mode, res_scale, _p(x_out), _ld(x_out), _p(w_pre),
                  _p(n_out), _ld(n_out), eps)
    _check("mxg_block_norm", load().mxg_block_norm(ctypes.byref(d), _s(stream)))


def mxg_block_norm_workspace_bytes(rows: int, cols: int) -> int:
    return load().mxg_block_norm_workspace_bytes(rows, cols)


def mxg_block_norm_backward(x: torch.Tensor, y=None, w_post=None, gate=None,
                            gate_mode: int = MXG_GATE_NONE, res_scale: float = 1.0, w_pre=None,
                            eps: float = 1e-6, dx_out=None, dn=None, dx=None, dy=None,
                            dw_post=None, dw_pre=None, dgate=None, workspace=None,
                            stream=None) -> None:
    """x: the block's output as mxg_block_norm stored it (x_out)."""
    rows, cols = x.shape
    full = gate_mode == MXG_GATE_FULL
    dtype = _same_type((y, dn, dy, w_post, w_pre, gate if gate_mode >= MXG_GATE_COL else None,
                        dgate if full else None))
    res = _same_type((x, dx_out, dx))
    _same_shape(x, (y, dx_out, dn, dx, dy))
    _vector(w_post, cols)
    _vector(w_pre, cols)
    _vector(dw_post, cols, True)
    _vector(dw_pre, cols, True)
    _gate(gate, gate_mode, x, False)
    _gate(dgate, gate_mode, x, True)
    d = BlockNormGrad(dtype, res, rows, cols, _p(x), _ld(x), _p(y), _ld(y), _p(w_post), _p(gate),
                      _ld(gate) if full else 0, gate_mode, res_scale, _p(w_pre), eps, _p(dx_out),
                      _ld(dx_out), _p(dn), _ld(dn), _p(dx), _ld(dx), _p(dy), _ld(dy), _p(dw_post),
                      _p(dw_pre), _p(dgate), _ld(dgate) if full else 0)
    _check("mxg_block_norm_backward",
           load().mxg_block_norm_backward(ctypes.byref(d), _p(_dense(workspace)),
                                          0 if workspace is None else workspace.nbytes, _s(stream)))


def mxg_grad_workspace_bytes() -> int:
    return load().mxg_grad_workspace_bytes()


class GradList:
    """An array of mxg_grad_t over tensors that it keeps alive (see grad_list)."""

    def __init__(self, src, dst):
        for t in (*src, *dst):
            if not t.is_contiguous() or t.dtype not in _DTYPES:
                raise ValueError("gradients are contiguous fp32, bf16 or fp16 tensors")
        if len(src) != len(dst) or any(s.numel() != d.numel() for s, d in zip(src, dst)):
            raise ValueError("one destination of the same size for each gradient")
        self.tensors = (tuple(src), tuple(dst))
        self.n = len(src)
        self.array = (Grad * max(1, self.n))(*[
            Grad(_p(s), _p(d), s.numel(), _DTYPES[s.dtype], _DTYPES[d.dtype])
            for s, d in zip(src, dst)])
        self.address = ctypes.addressof(self.array)


def grad_list(src, dst=None) -> GradList:
    """The list mxg_grad_norm and mxg_grad_clip take: gradients, and where their
    clipped values go (default: in place).  It can be used again as long as the
    gradients stay in the same tensors."""
    src = list(src)
    return GradList(src, src if dst is None else list(dst))


def mxg_grad_norm(grads: GradList, norm: torch.Tensor, workspace: torch.Tensor,
                  stream=None) -> None:
    assert norm.dtype == torch.float32
    _check("mxg_grad_norm",
           load().mxg_grad_norm(grads.address, grads.n, _p(norm), _p(_dense(workspace)),
                                workspace.nbytes, _s(stream)))


def mxg_grad_clip(grads: GradList, max_norm: float, norm: torch.Tensor, workspace: torch.Tensor,
                  stream=None) -> None:
    assert norm.dtype == torch.float32
    _check("mxg_grad_clip",
           load().mxg_grad_clip(grads.address, grads.n, max_norm, _p(norm), _p(_dense(workspace)),
                                workspace.nbytes, _s(stream)))


# ------------------------------------------------ around the products of an expert block
# A call of these takes 6 to 10 us of the host's time, of which every tensor's checks are some:
# they are made in one place, on the way to its address, and a descriptor is packed into bytes at
# once (a ctypes structure of 20 fields takes 2.5 us to fill).
_PACK = {ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}


def _packer(desc):
    """A function that packs a descriptor's fields, in their order, as C lays them out."""
    return struct.Struct("@" + "".join(_PACK[kind] for _, kind in desc._fields_)).pack


_pack_route, _pack_route_grad = _packer(Route), _packer(RouteGrad)
_pack_expert_rows, _pack_gated_act = _packer(ExpertRows), _packer(GatedAct)
_I32, _I64, _FP32 = (torch.int32,), (torch.int64,), (torch.float32,)
_MASK, _BYTES = (torch.uint8, torch.bool), (torch.uint8, torch.float8_e4m3fn)


# (the public torch.cuda.current_device takes twice the time)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here() -> int:
    """The device that launches go to."""
    return _device()


def _on(t, here: int) -> int:
    """The address of a tensor on the current device."""
    if t.get_device() != here:
        if not t.is_cuda:
            raise ValueError("libmxg takes device tensors; got a %s tensor" % t.device)
        raise ValueError("a tensor on %s: the current device is %d" % (t.device, here))
    return t.data_ptr()


def _whole(t, dtypes: tuple, n: int, name: str, here: int) -> int:
    """The address of a contiguous tensor of n elements of one of these types."""
    if t.dtype not in dtypes or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected %d contiguous elements of %s: got %s of %s"
                         % (name, n, dtypes[0], tuple(t.shape), t.dtype))
    return _on(t, here)


def _pitch(t, shape) -> int:
    """_ld of a [rows, cols] matrix, in a third of its time."""
    if t.is_contiguous():
        return 0
    rows, cols = shape
    between, within = t.stride()
    if (within != 1 and cols > 1) or (rows > 1 and between < cols):
        return _ld(t)  # which says what is wrong
    return between if rows > 1 else max(between, cols)


def _matrix(t, dtype, shape, name: str, here: int) -> tuple:
    """(address, elements between the rows) of a [rows, cols] matrix of this type; zeros of none."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError("%s: expected %s of %s: got %s of %s"
                         % (name, tuple(shape), dtype, tuple(t.shape), t.dtype))
    return _on(t, here), _pitch(t, shape)


def _workspace(t, here: int) -> tuple:
    """(address, bytes) of a workspace; zeros of none."""
    if t is None:
        return 0, 0
    return _on(_dense(t), here), t.nbytes


def _status(t, here: int) -> int:
    """The address of a status word (or the number that is given for one); 0 of none."""
    if t is None or isinstance(t, int):
        return t or 0
    if t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError("dev_status: expected an int32 word: got %s of %s"
                         % (tuple(t.shape), t.dtype))
    return _on(t, here)


def _stream_on(stream, here: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(here)
    return _s(stream)


def _choices(expert, name: str) -> tuple:
    """(tokens, k) of a [tokens, k] tensor of choices."""
    shape = expert.shape
    if len(shape) != 2:
        raise ValueError("%s: expected [tokens, k]: got %s" % (name, tuple(shape)))
    return shape


def _logits(t, tokens: int) -> tuple:
    """(type, experts) of the router's logits."""
    shape, kind = t.shape, _DTYPES.get(t.dtype)
    if len(shape) != 2 or shape[0] != tokens or kind is None:
        raise ValueError("logits: expected [%d, experts] of fp32, bf16 or fp16: got %s of %s"
                         % (tokens, tuple(shape), t.dtype))
    return kind, shape[1]


def _rows_wanted(row_of, group_ws, choices: int, experts: int, align: int, rows_capacity,
                 here: int) -> tuple:
    """(row_of, group_ws, capacity); the rows that always suffice where none are given."""
    if (row_of is None) != (group_ws is None):
        raise ValueError("row_of and group_ws: both or neither")
    if rows_capacity is None:
        rows_capacity = choices + experts * (align - 1)
    if row_of is None:
        return 0, 0, rows_capacity
    return (_whole(row_of, _I32, choices, "row_of", here),
            _whole(group_ws, _I64, 2 * experts + 1, "group_ws", here), rows_capacity)


def mxg_route_workspace_bytes(tokens: int, experts: int, k: int) -> int:
    return load().mxg_route_workspace_bytes(tokens, experts, k)


def mxg_route(logits: torch.Tensor, expert: torch.Tensor, weight: torch.Tensor,
              counts: torch.Tensor, mask=None, score: int = MXG_SCORE_SOFTMAX,
              normalize: bool = True, scale: float = 1.0, balance: float = 0.0, loss=None,
              slope=None, row_of=None, group_ws=None, align: int = 1, rows_capacity=None,
              last_dim: int = 1, workspace=None, dev_status=None, stream=None) -> None:
    """logits: [tokens, experts] (rows may be strided); expert, weight, row_of: [tokens, k];
    mask: uint8 or bool [tokens].  rows_capacity: by default the rows that always suffice,
    tokens * k + experts * (align - 1)."""
    here = _here()
    tokens, k = _choices(expert, "expert")
    kind, E = _logits(logits, tokens)
    n = tokens * k
    row, groups, capacity = _rows_wanted(row_of, group_ws, n, E, align, rows_capacity, here)
    d = _pack_route(kind, tokens, E, k, _on(logits, here), _pitch(logits, (tokens, E)),
                    0 if mask is None else _whole(mask, _MASK, tokens, "mask", here), score,
                    normalize, scale, balance, _whole(expert, _I32, n, "expert", here),
                    _whole(weight, _FP32, n, "weight", here), _whole(counts, _I32, E, "counts", here),
                    0 if loss is None else _whole(loss, _FP32, 1, "loss", here),
                    0 if slope is None else _whole(slope, _FP32, E, "slope", here), row, groups,
                    align, capacity, last_dim)
    ws, ws_bytes = _workspace(workspace, here)
    _check("mxg_route",
           load().mxg_route(d, ws, ws_bytes, _status(dev_status, here), _stream_on(stream, here)))


def mxg_route_rows(expert: torch.Tensor, counts: torch.Tensor, row_of=None, group_ws=None,
                   align: int = 1, rows_capacity=None, last_dim: int = 1, workspace=None,
                   dev_status=None, stream=None) -> None:
    """expert: int32 [tokens, k]; counts: int32 [experts]."""
    here = _here()
    tokens, k = _choices(expert, "expert")
    E, n = counts.numel(), tokens * k
    row, groups, capacity = _rows_wanted(row_of, group_ws, n, E, align, rows_capacity, here)
    ws, ws_bytes = _workspace(workspace, here)
    _check("mxg_route_rows",
           load().mxg_route_rows(_whole(expert, _I32, n, "expert", here), tokens, E, k, align,
                                 capacity, last_dim, _whole(counts, _I32, E, "counts", here), row,
                                 groups, ws, ws_bytes, _status(dev_status, here),
                                 _stream_on(stream, here)))


def mxg_route_backward(logits: torch.Tensor, expert: torch.Tensor, dlogits: torch.Tensor,
                       dweight=None, score: int = MXG_SCORE_SOFTMAX, normalize: bool = True,
                       scale: float = 1.0, slope=None, dloss=None, stream=None) -> None:
    """logits, expert, slope: as mxg_route took and wrote them; dlogits: like logits."""
    here = _here()
    tokens, k = _choices(expert, "expert")
    kind, E = _logits(logits, tokens)
    n = tokens * k
    d_at, ldd = _matrix(dlogits, logits.dtype, logits.shape, "dlogits", here)
    d = _pack_route_grad(kind, tokens, E, k, _on(logits, here), _pitch(logits, (tokens, E)),
                         _whole(expert, _I32, n, "expert", here), score, normalize, scale,
                         0 if dweight is None else _whole(dweight, _FP32, n, "dweight", here),
                         0 if slope is None else _whole(slope, _FP32, E, "slope", here),
                         0 if dloss is None else _whole(dloss, _FP32, 1, "dloss", here), d_at, ldd)
    _check("mxg_route_backward", load().mxg_route_backward(d, _stream_on(stream, here)))


def _expert_rows(fn: str, tokens, rows, row_of, weight, y_rows, dweight, counts, group_ws,
                 stream) -> None:
    here = _here()
    n, k = _choices(row_of, "row_of")
    shape, dtype = tokens.shape, tokens.dtype
    kind = _DTYPES.get(dtype)
    if len(shape) != 2 or shape[0] != n or kind is None:
        raise ValueError("expected [%d, cols] of fp32, bf16 or fp16: got %s of %s"
                         % (n, tuple(shape), dtype))
    cols, like = shape[1], y_rows if rows is None else rows
    if like is None:
        raise ValueError("%s: no rows are given" % fn)
    capacity = like.shape[0]
    rows_at, ldr = _matrix(rows, dtype, (capacity, cols), "rows", here)
    y_at, ldy = _matrix(y_rows, dtype, (capacity, cols), "y_rows", here)
    if (counts is None) != (group_ws is None):
        raise ValueError("counts and group_ws: both or neither")
    experts = 0 if counts is None else counts.numel()
    at = _whole(row_of, _I32, n * k, "row_of", here)
    w_at = 0 if weight is None else _whole(weight, _FP32, n * k, "weight", here)
    dw_at = 0 if dweight is None else _whole(dweight, _FP32, n * k, "dweight", here)
    c_at = g_at = 0
    if counts is not None:
        c_at = _whole(counts, _I32, experts, "counts", here)
        g_at = _whole(group_ws, _I64, 2 * experts + 1, "group_ws", here)
    d = _pack_expert_rows(kind, n, cols, k, experts, capacity, _on(tokens, here),
                          _pitch(tokens, shape), rows_at, ldr, at, w_at, y_at, ldy, dw_at, c_at, g_at)
    _check(fn, getattr(load(), fn)(d, _stream_on(stream, here)))


def mxg_dispatch(tokens: torch.Tensor, row_of: torch.Tensor, rows: torch.Tensor, counts=None,
                 group_ws=None, stream=None) -> None:
    """tokens [n, cols] to rows [rows_capacity, cols] (rows of both may be strided); counts and
    group_ws: to set the groups' padding rows to 0."""
    _expert_rows("mxg_dispatch", tokens, rows, row_of, None, None, None, counts, group_ws, stream)


def mxg_combine(rows: torch.Tensor, row_of: torch.Tensor, tokens: torch.Tensor, weight=None,
                stream=None) -> None:
    """tokens[t] = the sum of rows[row_of[t, j]], times weight[t, j] where that is given."""
    _expert_rows("mxg_combine", tokens, rows, row_of, weight, None, None, None, None, stream)


def mxg_combine_backward(dtokens: torch.Tensor, row_of: torch.Tensor, weight, drows, y_rows=None,
                         dweight=None, counts=None, group_ws=None, stream=None) -> None:
    """The gradients drows of the rows and dweight of the weights (either may be None); y_rows:
    the rows that mxg_combine summed, for dweight."""
    if drows is None and dweight is None:
        raise ValueError("drows, dweight: one of them at least")
    _expert_rows("mxg_combine_backward", dtokens, drows, row_of, weight, y_rows, dweight, counts,
                 group_ws, stream)


def _act_blocks(cols: int) -> int:
    return (cols + 31) // 32


def _kept(q, sf, rows: int, cols: int, parts: int, here: int) -> tuple:
    """(q, bytes between its rows, sf) of an 8-bit checkpoint of `parts` matrices, or zeros."""
    if (q is None) != (sf is None):
        raise ValueError("q and sf: both or neither")
    if q is None:
        return 0, 0, 0
    if q.dtype not in _BYTES or q.shape != (rows, parts * cols):
        raise ValueError("q: expected %s bytes: got %s of %s"
                         % ((rows, parts * cols), tuple(q.shape), q.dtype))
    return (_on(q, here), _pitch(q, (rows, parts * cols)),
            _whole(sf, _BYTES[:1], rows * parts * _act_blocks(cols), "sf", here))


def _act_shape(t, name: str) -> tuple:
    """(type, rows, cols)"""
    shape, kind = t.shape, _DTYPES.get(t.dtype)
    if len(shape) != 2 or kind is None:
        raise ValueError("%s: expected [rows, cols]: got %s of %s" % (name, tuple(shape), t.dtype))
    return kind, shape[0], shape[1]


def mxg_gated_act(gate: torch.Tensor, h: torch.Tensor, up=None, act: int = MXG_ACT_SILU, q=None,
                  sf=None, group_ws=None, G: int = 0, stream=None) -> None:
    """h = act(gate) * up, [rows, cols] (rows may be strided: gate and up are often the halves of
    one product); q, sf: where the inputs are kept (alloc_act_checkpoint)."""
    here = _here()
    kind, rows, cols = _act_shape(gate, "gate")
    parts = 1 if up is None else 2
    up_at, ldu = _matrix(up, gate.dtype, gate.shape, "up", here)
    h_at, ldh = _matrix(h, gate.dtype, gate.shape, "h", here)
    q_at, ldq, sf_at = _kept(q, sf, rows, cols, parts, here)
    d = _pack_gated_act(kind, act, rows, cols, parts - 1, G,
                        0 if group_ws is None else _whole(group_ws, _I64, 2 * G + 1, "group_ws", here),
                        _on(gate, here), _pitch(gate, (rows, cols)),
                        up_at, ldu, h_at, ldh, q_at, ldq, sf_at, 0, 0, 0, 0, 0, 0)
    _check("mxg_gated_act", load().mxg_gated_act(d, _stream_on(stream, here)))


def mxg_gated_act_backward(q: torch.Tensor, sf: torch.Tensor, dh: torch.Tensor, dgate: torch.Tensor,
                           dup=None, act: int = MXG_ACT_SILU, h=None, group_ws=None, G: int = 0,
                           stream=None) -> None:
    """The gradients of gate and up from the checkpoint, and h again where it is given."""
    here = _here()
    kind, rows, cols = _act_shape(dh, "dh")
    parts = 1 if dup is None else 2
    dgate_at, lddg = _matrix(dgate, dh.dtype, dh.shape, "dgate", here)
    dup_at, lddu = _matrix(dup, dh.dtype, dh.shape, "dup", here)
    h_at, ldh = _matrix(h, dh.dtype, dh.shape, "h", here)
    q_at, ldq, sf_at = _kept(q, sf, rows, cols, parts, here)
    d = _pack_gated_act(kind, act, rows, cols, parts - 1, G,
                        0 if group_ws is None else _whole(group_ws, _I64, 2 * G + 1, "group_ws", here),
                        0, 0, 0, 0, h_at, ldh, q_at,
                        ldq, sf_at, _on(dh, here), _pitch(dh, (rows, cols)), dgate_at, lddg, dup_at, lddu)
    _check("mxg_gated_act_backward", load().mxg_gated_act_backward(d, _stream_on(stream, here)))


def mxg_status_string(code: int) -> str:
    return load().mxg_status_string(code).decode()


def mxg_version() -> int:
    return load().mxg_version()


def mxg_launch_count() -> int:
    return load().mxg_launch_count()


# ----------------------------------------------------------------- buffer helpers
def alloc_offsets(G: int, device="cuda") -> torch.Tensor:
    return torch.empty(2 * G + 1, dtype=torch.int64, device=device)


def alloc_mxfp8(rows: int, cols: int, rowwise=True, colwise=False, device="cuda") -> dict:
    out = {}
    if rowwise:
        out["q_row"] = torch.empty((rows, cols), dtype=torch.uint8, device=device)
        out["sf_row"] = torch.empty(rows * cols // 32, dtype=torch.uint8, device=device)
    if colwise:
        out["q_col"] = torch.empty((cols, rows), dtype=torch.uint8, device=device)
        out["sf_col"] = torch.empty(rows * cols // 32, dtype=torch.uint8, device=device)
    return out


def alloc_mxfp8_unaligned(rows: int, cols: int, G: int, rowwise=True, colwise=False,
                          device="cuda") -> dict:
    """Buffers for mxg_group_quantize_unaligned: dense rowwise data, scales and
    colwise copy over the padded row count rows + 128 G."""
    rp = rows + 128 * G
    out = {}
    if rowwise:
        out["q_row"] = torch.empty((rows, cols), dtype=torch.uint8, device=device)
        out["sf_row"] = torch.empty(rp * cols // 32, dtype=torch.uint8, device=device)
    if colwise:
        out["q_col"] = torch.empty((cols, rp), dtype=torch.uint8, device=device)
        out["sf_col"] = torch.empty(rp * cols // 32, dtype=torch.uint8, device=device)
    return out


def alloc_nvfp4(rows: int, cols: int, device="cuda", rowwise=True, colwise=False,
                G: int = 1) -> dict:
    out = {}
    if rowwise:
        out["q_row"] = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        out["sf_row"] = torch.empty(rows * cols // 16, dtype=torch.uint8, device=device)
        out["outer_row"] = torch.empty(rows, dtype=torch.float32, device=device)
    if colwise:
        out["q_col"] = torch.empty((cols, rows // 2), dtype=torch.uint8, device=device)
        out["sf_col"] = torch.empty(rows * cols // 16, dtype=torch.uint8, device=device)
        out["outer_col"] = torch.empty((G, cols), dtype=torch.float32, device=device)
    return out


def alloc_block_norm_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(16, mxg_block_norm_workspace_bytes(rows, cols)), dtype=torch.uint8,
                       device=device)


def alloc_grad_workspace(device="cuda") -> torch.Tensor:
    return torch.empty(mxg_grad_workspace_bytes(), dtype=torch.uint8, device=device)


def alloc_route_workspace(tokens: int, experts: int, k: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(16, mxg_route_workspace_bytes(tokens, experts, k)), dtype=torch.uint8,
                       device=device)


def alloc_act_checkpoint(rows: int, cols: int, gated: bool = True, device="cuda") -> tuple:
    """(q, sf) of mxg_gated_act: E4M3 bytes of gate and up side by side, and their scales."""
    parts = 2 if gated else 1
    return (torch.empty((rows, parts * cols), dtype=torch.uint8, device=device),
            torch.empty((rows, parts * _act_blocks(cols)), dtype=torch.uint8, device=device))
