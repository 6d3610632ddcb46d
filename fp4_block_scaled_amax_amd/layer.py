"""Python binding of libue5m3fp4_layer: the operators next to the FP4 linears.

  * the 8-bit linear: quantize_fp8 and gemm_fp8_fprop / _dgrad / _wgrad on
    E4M3 / E5M2 codes with one scale per block of 128, for the linears that
    the FP4 recipe leaves in higher precision;
  * dropout and dropout_backward: a counter-based mask that is never stored,
    the residual addition and the running amax of the periodic tensor scale.

Argument marshalling only, as in the package itself; the C ABI, the layouts
and the exact arithmetic are documented in include/ue5m3fp4_layer.h.  Every
function launches on the device of its tensors, on torch's current stream of
that device unless one is given.
"""

import ctypes
import os
from dataclasses import dataclass

from . import _check, _i64, _PKG, _require, _require_scalar, _same_device

LAYER_LIB_PATH = os.path.join(_PKG, "libue5m3fp4_layer.so")

E4M3 = 0
E5M2 = 1
FP8_BLOCK = 128

_void = ctypes.c_void_p
_int = ctypes.c_int
_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32

_SIGNATURES = {
    "ue5m3fp4_quantize_fp8": [_void, _i64, _i64, _i64, _int, _int, _int, _void, _void, _void, _void, _void],
    "ue5m3fp4_gemm_fp8_nt": [_void, _void, _int, _int, _void, _void, _int, _int, _int, _i64, _i64, _i64, _void, _int,
                             _void],
    "ue5m3fp4_dropout": [_void, _int, _i64, _void, _i64, _void, _int, _i64, _i64, _i64, ctypes.c_double, _u64, _u32,
                         _void, _void],
    "ue5m3fp4_dropout_backward": [_void, _int, _i64, _void, _int, _i64, _i64, _i64, ctypes.c_double, _u64, _u32,
                                  _void, _void],
}

_lib = None


def load_layer_library(path=LAYER_LIB_PATH):
    """Load libue5m3fp4_layer.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m fp4_block_scaled_amax_amd.build` (needs hipcc)")
    lib = ctypes.CDLL(path)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    _lib = lib
    return lib


def _launch(where, device, stream, *args):
    """Call the entry point `where` with `args` and the stream, with `device` current."""
    import torch

    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    elif getattr(stream, "device", device) != device:
        raise ValueError(f"{where}: the stream belongs to {stream.device}, the tensors are on {device}")
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    fn = getattr(_lib or load_layer_library(), where)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != 0:
        _check(status, where)


def _device_of(where, *tensors):
    """The device that all the tensors (or None) share."""
    device = tensors[0].device
    for t in tensors:
        if t is not None and t.device != device:
            _same_device(where, *tensors)
    return device


def _address(t):
    return None if t is None else t.data_ptr()


def _blocks(n):
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


@dataclass
class Fp8Quantized:
    """One 8-bit operand of `cols` columns, blocked along them: codes
    [R][cols rounded up to 128] uint8; scales fp32, or uint8 for E8M0,
    [blocks of cols][R] or, for 128 x 128 tiles, [blocks of cols][blocks of R]."""

    codes: "object"
    scales: "object"
    cols: int
    fmt: int = E4M3
    tile: bool = False

    @property
    def rows(self):
        return self.codes.shape[0]


def empty_quantized_fp8(rows, cols, fmt=E4M3, e8m0=False, tile=False, device="cuda"):
    """Allocate the code and scale buffers of a rows x cols 8-bit operand."""
    import torch

    return Fp8Quantized(torch.empty((rows, _blocks(cols) * FP8_BLOCK), dtype=torch.uint8, device=device),
                        torch.empty((_blocks(cols), _blocks(rows) if tile else rows),
                                    dtype=torch.uint8 if e8m0 else torch.float32, device=device), cols, fmt, tile)


def _check_fp8(q, name):
    """An Fp8Quantized operand with contiguous device buffers of its shapes."""
    import torch

    if not isinstance(q, Fp8Quantized):
        raise ValueError(f"{name} must be an Fp8Quantized operand")
    if q.fmt not in (E4M3, E5M2):
        raise ValueError(f"{name}: unknown format {q.fmt}")
    if q.cols < 0:
        raise ValueError(f"{name}: cols is negative")
    _require(q.codes, (torch.uint8,), name + " codes", 2, contiguous=True)
    _require(q.scales, (torch.float32, torch.uint8), name + " scales", 2, contiguous=True)
    rows, padded = q.codes.shape
    blocks = _blocks(q.cols)
    if padded != blocks * FP8_BLOCK:
        raise ValueError(f"{name}: codes {tuple(q.codes.shape)} do not match {q.cols} columns "
                         f"([{rows}][{blocks * FP8_BLOCK}])")
    if q.scales.shape != (blocks, _blocks(rows) if q.tile else rows):
        raise ValueError(f"{name}: scales {tuple(q.scales.shape)} do not match a {rows} x {q.cols} operand "
                         f"([{blocks}][{_blocks(rows) if q.tile else rows}])")
    return rows


def _matrix(t, name):
    """(rows, cols, row stride) of a 2-D tensor with unit stride along its columns."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its columns")
    return rows, cols, t.stride(0) if rows > 1 else cols


def quantize_fp8(x, row=None, col=None, stream=None):
    """Quantize a bf16 (rows x cols) tensor to 8 bits.  row: the operand
    blocked along cols (rows x cols); col: x^T blocked along rows (cols x
    rows), from the same read; at least one.  Format, scale type (the dtype of
    `scales`) and tile mode are those of the outputs, which must agree."""
    import torch

    _require(x, (torch.bfloat16, torch.int16, torch.uint16), "x", 2)
    rows, cols, ld = _matrix(x, "x")
    outs = [(o, n, r, c) for o, n, r, c in ((row, "row", rows, cols), (col, "col", cols, rows)) if o is not None]
    if not outs:
        raise ValueError("quantize_fp8: row or col is required")
    for o, n, r, c in outs:
        if (_check_fp8(o, n), o.cols) != (r, c):
            raise ValueError(f"{n} is a {o.rows} x {o.cols} operand, expected {r} x {c}")
    q = outs[0][0]
    if len(outs) == 2 and (row.fmt, row.tile, row.scales.dtype) != (col.fmt, col.tile, col.scales.dtype):
        raise ValueError("row and col disagree on format, tile mode or scale type")
    buffers = [t for o in (row, col) for t in ((o.codes, o.scales) if o is not None else (None, None))]
    device = _device_of("quantize_fp8", x, *buffers)
    _launch("ue5m3fp4_quantize_fp8", device, stream, x.data_ptr(), rows, cols, ld, q.fmt,
            int(q.scales.dtype == torch.uint8), int(q.tile), *map(_address, buffers))


def _gemm_fp8(a, b, out, stream, na, nb):
    import torch

    M, N, K = _check_fp8(a, na), _check_fp8(b, nb), a.cols
    if K != b.cols:
        raise ValueError(f"{na} and {nb} disagree on the contraction axis ({K} vs {b.cols})")
    if a.scales.dtype != b.scales.dtype:
        raise ValueError(f"{na} and {nb} have scales of different types")
    _require(out, (torch.float32, torch.bfloat16), "out", 2, contiguous=True)
    if out.shape != (M, N):
        raise ValueError(f"output must be a contiguous [{M}][{N}] tensor")
    device = _device_of("gemm_fp8", out, a.codes, a.scales, b.codes, b.scales)
    _launch("ue5m3fp4_gemm_fp8_nt", device, stream, a.codes.data_ptr(), a.scales.data_ptr(), a.fmt, int(a.tile),
            b.codes.data_ptr(), b.scales.data_ptr(), b.fmt, int(b.tile), int(a.scales.dtype == torch.uint8), M, N, K,
            out.data_ptr(), int(out.dtype == torch.float32))
    return out


def gemm_fp8_nt(a, b, out, stream=None):
    """out[M][N] = A B^T of two 8-bit operands blocked along K.  An fp32 out has
    exact products and fp32 sums; a bf16 out runs twice as fast on the 8-bit
    matrix instructions, which keep of each 8 products what lies within 2^-13
    of the largest (1e-5 to 1e-4 of the result's norm, and at most 2^-10 sum
    |a b| of an entry, before the rounding to bf16)."""
    return _gemm_fp8(a, b, out, stream, "A", "B")


def gemm_fp8_fprop(x_row, w_row, y, stream=None):
    """Y [tokens][out] = X W^T from X and W quantized row-wise (y's type: see gemm_fp8_nt)."""
    return _gemm_fp8(x_row, w_row, y, stream, "x_row", "w_row")


def gemm_fp8_dgrad(dy_row, w_col, dx, stream=None):
    """dX [tokens][in] = dY W from dY row-wise and W's transposed output (dx's type: see gemm_fp8_nt)."""
    return _gemm_fp8(dy_row, w_col, dx, stream, "dy_row", "w_col")


def gemm_fp8_wgrad(dy_col, x_col, dw, stream=None):
    """dW [out][in] = dY^T X from the transposed outputs of dY and X (dw's type: see gemm_fp8_nt)."""
    return _gemm_fp8(dy_col, x_col, dw, stream, "dy_col", "x_col")


def _flat(t, name, cols):
    """Row stride of a tensor taken as a matrix of `cols` columns."""
    if t.is_contiguous():
        return cols
    if t.dim() != 2:
        raise ValueError(f"{name} must be contiguous, or a matrix with unit stride along its columns")
    return _matrix(t, name)[2]


def _dropout(where, x, p, seed, offset, out, residual, amax, stream, nx, nout):
    import torch

    types = (torch.bfloat16, torch.float32)
    _require(x, types, nx)
    _require(out, types, nout)
    shape = x.shape
    if out.shape != shape:
        raise ValueError(f"{nout} has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if residual is not None:
        _require(residual, (out.dtype,), "residual")
        if residual.shape != shape:
            raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {tuple(shape)}")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must lie in [0, 1] (got {p})")
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 32:
        raise ValueError("seed must fit 64 unsigned bits and offset 32")
    if amax is not None:
        _require_scalar(amax, "amax")
    device = _device_of("dropout", x, out, residual, amax)
    rows, cols = shape if len(shape) == 2 else (1, x.numel())
    f32 = torch.float32
    args = [x.data_ptr(), int(x.dtype == f32), _flat(x, nx, cols)]
    if where == "ue5m3fp4_dropout":
        args += [_address(residual), _flat(residual, "residual", cols) if residual is not None else 0]
    _launch(where, device, stream, *args, out.data_ptr(), int(out.dtype == f32), _flat(out, nout, cols), rows, cols,
            float(p), int(seed), int(offset), _address(amax))
    return out


def dropout(x, p, seed, offset, out, residual=None, amax=None, stream=None):
    """out = residual + dropout(x): each element of x (bf16 or fp32) is zeroed
    with probability p (to the nearest multiple of 2^-16) or scaled by 1 / (1
    - p), by the counter-based stream (seed, offset), which are values of the
    call: a captured graph repeats its mask at every replay.  residual: of
    out's type, or None.  amax (device fp32 scalar or None) receives max(amax, max|out|).
    Tensors of one shape: contiguous, of any dimension and below 2^40 elements,
    or matrices (below 2^31 rows) with unit column stride."""
    return _dropout("ue5m3fp4_dropout", x, p, seed, offset, out, residual, amax, stream, "x", "out")


def dropout_backward(dy, p, seed, offset, dx, amax=None, stream=None):
    """dx: the gradient of dropout's x for the same (p, seed, offset) and
    shape; the mask is drawn again.  (The residual's gradient is dy.)"""
    return _dropout("ue5m3fp4_dropout_backward", dy, p, seed, offset, dx, None, amax, stream, "dy", "dx")
