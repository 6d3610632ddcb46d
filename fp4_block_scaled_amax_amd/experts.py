"""Python binding of libue5m3fp4_experts: the FP4 linears of routed experts.

  * quantize_grouped: rows grouped by expert (gathered by an index, if given)
    to the row-wise and the grouped transposed operand;
  * gemm_grouped_fprop / _dgrad / _wgrad: the experts' training GEMMs;
  * gemm_weight_only: bf16 tokens times FP4 weights, dense or of experts, for
    the few tokens of a generation step.

The rows of a grouped matrix are sorted by expert; `offsets`, a device int32
tensor of experts + 1 values, says which rows are whose: expert g owns rows
offsets[g] .. offsets[g + 1] - 1.  Its values stay on the device.

Argument marshalling only, as in the package itself; the C ABI, the layouts
and the arithmetic are documented in include/ue5m3fp4_experts.h.  Every
function launches on the device of its tensors, on torch's current stream of
that device unless one is given.
"""

import ctypes
import os
from dataclasses import dataclass

from . import RNE, Quantized, _check_operand, _check_pair, _i64, _PKG, _require, _require_scalar
from .layer import _address, _enqueue, _matrix

EXPERTS_LIB_PATH = os.path.join(_PKG, "libue5m3fp4_experts.so")

_void = ctypes.c_void_p
_int = ctypes.c_int

_SIGNATURES = {
    "ue5m3fp4_quantize_grouped": [_void, _i64, _i64, _i64, _void, _i64, _void, _i64, _void, _int, ctypes.c_uint64,
                                  ctypes.c_uint32, _void, _void, _void, _void, _void, _void],
    "ue5m3fp4_gemm_grouped_nt": [_void] * 6 + [_i64, _void, _i64, _i64, _i64, _i64, _void, _int, _void, _void],
    "ue5m3fp4_gemm_grouped_wgrad": [_void] * 7 + [_i64, _i64, _i64, _i64, _void, _int, _void],
    "ue5m3fp4_gemm_weight_only": [_void, _i64, _void, _void, _void, _i64, _void, _i64, _i64, _i64, _i64, _void, _int,
                                  _i64, _void],
}

_lib = None


def load_experts_library(path=EXPERTS_LIB_PATH):
    """Load libue5m3fp4_experts.so (once).  Raises if it has not been built."""
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
    """Call the entry point `where` of this library."""
    _enqueue(getattr(_lib or load_experts_library(), where), where, device, stream, *args)


@dataclass
class ExpertWeights:
    """Block-scaled operands of all experts: codes [experts][R][C/2] uint8,
    scales [experts][R][C/16] uint8, ts = device fp32 tensor scales (1 element
    for all experts, or one for each).  Blocks run along C."""

    codes: "object"
    scales: "object"
    ts: "object"

    @property
    def experts(self):
        return self.codes.shape[0]

    def expert(self, g):
        """Expert g's operand (views), for gemm_weight_only, and as an output of quantize_blockscale or an operand of
        the other products where R * C / 16 is a multiple of 16 (they need 16-byte aligned scales)."""
        g = range(self.experts)[g]
        return Quantized(self.codes[g], self.scales[g], self.ts[g:g + 1] if self.ts.numel() > 1 else self.ts)


def empty_expert_weights(experts, rows, cols, ts, device=None):
    """Allocate the code and scale buffers of one rows x cols operand per expert."""
    import torch

    device = device if device is not None else ts.device
    return ExpertWeights(torch.empty((experts, rows, cols // 2), dtype=torch.uint8, device=device),
                         torch.empty((experts, rows, cols // 16), dtype=torch.uint8, device=device), ts)


def rows_padded(rows, experts):
    """Columns of the grouped transposed operand of `rows` rows: expert g's
    stand from column 128 * (ceil(offsets[g] / 128) + g) on."""
    return 128 * ((rows + 127) // 128 + experts)


# The checks below ask each tensor once for what they need, since a call of a
# generation step lasts little longer than its checks, and leave the messages
# to _require and its like where something is wrong.


def _buffer(t, dtype, dims, device, name):
    """Shape of a contiguous `dims`-dimensional tensor of `dtype` on `device`."""
    try:
        shape = t.shape
        if t.dtype is dtype and t.device == device and len(shape) == dims and t.is_contiguous():
            return shape
    except AttributeError:
        pass
    _require(t, (dtype,), name, dims, contiguous=True)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _scalar(t, device, name):
    """A device fp32 scalar on `device`."""
    _require_scalar(t, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t, dtypes, name):
    """(rows, cols, row stride, device) of a 2-D device tensor with unit stride along its columns."""
    try:
        if t.is_cuda and t.dtype in dtypes:
            (rows, cols), (ld, unit) = t.shape, t.stride()
            if unit == 1 or cols <= 1:
                return rows, cols, ld if rows > 1 else cols, t.device
    except (AttributeError, ValueError, TypeError):
        pass
    _require(t, dtypes, name, 2)
    return (*_matrix(t, name), t.device)


def _experts(offsets, device):
    """Number of experts of an offsets tensor."""
    import torch

    n = _buffer(offsets, torch.int32, 1, device, "offsets")[0]
    if n < 1:
        raise ValueError("offsets must hold experts + 1 values")
    return n - 1


def _operand(q, device, name):
    """(rows, cols) of a Quantized operand."""
    import torch

    if not isinstance(q, Quantized):
        raise ValueError(f"{name} must be a Quantized operand")
    rows, half = _buffer(q.codes, torch.uint8, 2, device, name)
    if half % 8 != 0 or _buffer(q.scales, torch.uint8, 2, device, name) != (rows, half // 8):
        _check_operand(q, name)
    if q.ts.dtype is not torch.float32 or q.ts.numel() != 1 or q.ts.device != device:
        _scalar(q.ts, device, f"{name} ts")
    return rows, 2 * half


def _weights(w, experts, device, name):
    """(rows, cols) of one expert's operand in an ExpertWeights."""
    import torch

    if not isinstance(w, ExpertWeights):
        raise ValueError(f"{name} must be an ExpertWeights operand")
    n, rows, half = _buffer(w.codes, torch.uint8, 3, device, name)
    if n != experts:
        raise ValueError(f"{name} holds {n} experts, offsets {experts}")
    if half % 8 != 0 or _buffer(w.scales, torch.uint8, 3, device, name) != (n, rows, half // 8):
        raise ValueError(f"{name}: codes {tuple(w.codes.shape)} / scales {tuple(w.scales.shape)} do not match "
                         "([experts][R][C/2], [experts][R][C/16], C a multiple of 16)")
    if _buffer(w.ts, torch.float32, 1, device, name)[0] not in (1, n):
        raise ValueError(f"{name}: ts must hold 1 value or one per expert (has {w.ts.numel()})")
    return rows, 2 * half


def _result(out, device, shape, name="out"):
    """Whether a contiguous result tensor of this shape is fp32 (else bf16)."""
    import torch

    f32 = out.dtype is torch.float32
    if _buffer(out, torch.float32 if f32 else torch.bfloat16, len(shape), device, name) != shape:
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor (has {list(out.shape)})")
    return f32


def _device(t, name):
    if t is None or not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a device (cuda) tensor")
    return t.device


def quantize_grouped(x, offsets, tensor_scale, rounding=RNE, seed=0, offset=0, row=None, col=None, index=None,
                     amax=None, stream=None):
    """Quantize bf16 rows grouped by expert.  The grouped matrix is x, or with
    index (device int32) row i is x[index[i]]; an index out of range gives a
    row of zeros.  row: Quantized (rows x cols); col: Quantized grouped
    transposed operand (cols x rows_padded(rows, experts)); amax: device fp32
    scalar that receives max(amax, max|x|) over the experts' rows; at least one
    of the three.  Rows of no expert, and columns of col that are no expert's
    padding, keep what they held."""
    import torch

    x_rows, cols, ld, device = _rows(x, (torch.bfloat16, torch.int16, torch.uint16), "x")
    experts, rows = _experts(offsets, device), x_rows
    if index is not None:
        rows = _buffer(index, torch.int32, 1, device, "index")[0]
    buffers = []
    for q, name, r, c in ((row, "row output", rows, cols), (col, "col output", cols, rows_padded(rows, experts))):
        if q is None:
            buffers += [None, None]
            continue
        codes, scales = (q.codes, q.scales) if isinstance(q, Quantized) else q
        if (_buffer(codes, torch.uint8, 2, device, name) != (r, c // 2)
                or _buffer(scales, torch.uint8, 2, device, name) != (r, c // 16)):
            _check_pair(codes, scales, r, c, name)
        buffers += [codes, scales]
    if row is None and col is None and amax is None:
        raise ValueError("quantize_grouped: row, col or amax is required")
    if tensor_scale is not None:
        _scalar(tensor_scale, device, "tensor_scale")
    elif row is not None or col is not None:
        raise ValueError("tensor_scale is required")
    if amax is not None:
        _scalar(amax, device, "amax")
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 32:
        raise ValueError("seed must fit 64 unsigned bits and offset 32")
    _launch("ue5m3fp4_quantize_grouped", device, stream, x.data_ptr(), x_rows, cols, ld, _address(index), rows,
            offsets.data_ptr(), experts, _address(tensor_scale), int(rounding), int(seed), int(offset),
            *map(_address, buffers), _address(amax))


def _gemm_grouped(a, w, offsets, out, amax, stream, na, nw):
    device = _device(out, "out")
    experts = _experts(offsets, device)
    (rows, ak), (N, K) = _operand(a, device, na), _weights(w, experts, device, nw)
    if ak != K:
        raise ValueError(f"{na} and {nw} disagree on the contraction axis ({ak} vs {K})")
    f32 = _result(out, device, (rows, N))
    if amax is not None:
        _scalar(amax, device, "amax")
        if f32:
            raise ValueError("amax is for bf16 outputs")
    _launch("ue5m3fp4_gemm_grouped_nt", device, stream, a.codes.data_ptr(), a.scales.data_ptr(), a.ts.data_ptr(),
            w.codes.data_ptr(), w.scales.data_ptr(), w.ts.data_ptr(), w.ts.numel(), offsets.data_ptr(), experts,
            rows, N, K, out.data_ptr(), f32, _address(amax))
    return out


def gemm_grouped_fprop(x_row, w_row, offsets, y, amax=None, stream=None):
    """Y [rows][out] (bf16 or fp32): rows of expert g times W_g^T, from X
    row-wise (grouped) and ExpertWeights W [experts][out][in].  amax (bf16 Y
    only) receives max(amax, max|Y|).  Rows of no expert keep what they held."""
    return _gemm_grouped(x_row, w_row, offsets, y, amax, stream, "x_row", "w_row")


def gemm_grouped_dgrad(dy_row, w_col, offsets, dx, amax=None, stream=None):
    """dX [rows][in] (bf16 or fp32): rows of expert g times W_g, from dY row-wise
    and the experts' transposed outputs W^T [experts][in][out]."""
    return _gemm_grouped(dy_row, w_col, offsets, dx, amax, stream, "dy_row", "w_col")


def gemm_grouped_wgrad(dy_col, x_col, offsets, dw, stream=None, rows=None):
    """dW [experts][out][in] (bf16 or fp32) = dY^T X over each expert's rows,
    from the grouped transposed operands of dY and X; zeros for an expert
    without rows.  rows: how many the operands were quantized from, to which
    offsets past them are clamped as they were there.  Their columns tell it up
    to a multiple of 128 alone, so it is needed where offsets may pass the rows;
    where they do not, it changes nothing."""
    device = _device(dw, "dw")
    experts = _experts(offsets, device)
    (M, padded), (N, x_padded) = _operand(dy_col, device, "dy_col"), _operand(x_col, device, "x_col")
    whole = padded - 128 * experts
    if rows is None:
        rows = whole
    if rows < 0 or whole % 128 != 0 or whole != 128 * ((rows + 127) // 128) or x_padded != padded:
        raise ValueError(f"dy_col and x_col must have rows_padded(rows, {experts}) columns "
                         f"(have {padded} and {x_padded})")
    f32 = _result(dw, device, (experts, M, N), "dw")
    _launch("ue5m3fp4_gemm_grouped_wgrad", device, stream, dy_col.codes.data_ptr(), dy_col.scales.data_ptr(),
            dy_col.ts.data_ptr(), x_col.codes.data_ptr(), x_col.scales.data_ptr(), x_col.ts.data_ptr(),
            offsets.data_ptr(), experts, rows, M, N, dw.data_ptr(), f32)
    return dw


def gemm_weight_only(x, w, out, offsets=None, stream=None):
    """out [rows][N] (bf16 or fp32, unit column stride) = x W^T with x [rows][K]
    in bf16 and FP4 weights: w a Quantized [N][K], or with offsets the
    ExpertWeights [experts][N][K] of the rows' experts.  Made for few rows (1 to
    about 64 per expert).  Rows of no expert keep what they held."""
    import torch

    rows, K, ldx, device = _rows(x, (torch.bfloat16, torch.int16, torch.uint16), "x")
    if offsets is None:
        experts, (N, wk) = 1, _operand(w, device, "w")
    else:
        experts = _experts(offsets, device)
        N, wk = _weights(w, experts, device, "w")
    if wk != K:
        raise ValueError(f"x and w disagree on the contraction axis ({K} vs {wk})")
    out_rows, out_cols, ldo, out_device = _rows(out, (torch.bfloat16, torch.float32), "out")
    if out_rows != rows or out_cols != N:
        raise ValueError(f"out must be a [{rows}][{N}] tensor (has {list(out.shape)})")
    if out_device != device:
        raise ValueError(f"out is on {out_device}, x on {device}")
    _launch("ue5m3fp4_gemm_weight_only", device, stream, x.data_ptr(), ldx, w.codes.data_ptr(), w.scales.data_ptr(),
            w.ts.data_ptr(), w.ts.numel(), _address(offsets), experts, rows, N, K, out.data_ptr(),
            out.dtype is torch.float32, ldo)
    return out
