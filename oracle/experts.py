"""The linears of routed experts (oracle side).

TEST INFRASTRUCTURE: see oracle/__init__.py for who may use this module.

[UE5M3] abstract: FP4 in all eligible internal linears; an expert's linears are
ordinary linears over the rows that were routed to it, so each is quantize.py's
and gemm.py's definition on its own rows.  Reading: the rows are sorted by
expert, expert g owns rows offsets[g] .. offsets[g + 1] - 1; in a transposed
operand they begin at column 128 (ceil(offsets[g] / 128) + g) and are followed
by zeros up to the next multiple of 128, so no block of 16 spans two experts.
Stochastic rounding counts the elements of that operand.

Everything is a loop over experts around the definitions for one matrix.
"""

import numpy as np

from . import formats, gemm, quantize


def rows_padded(rows, experts):
    return 128 * (-(-rows // 128) + experts)


def spans(offsets):
    """(first row, rows, first column of the transposed operand, columns with padding) of each expert."""
    out = []
    for g in range(len(offsets) - 1):
        b, n = int(offsets[g]), int(offsets[g + 1]) - int(offsets[g])
        out.append((b, n, 128 * (-(-b // 128) + g), -(-n // 128) * 128))
    return out


def gather(x_bits, index):
    """Rows x[index]; zeros where the index is out of range."""
    if index is None:
        return x_bits
    out = np.zeros((len(index), x_bits.shape[1]), dtype=np.uint16)
    for i, j in enumerate(index):
        if 0 <= j < x_bits.shape[0]:
            out[i] = x_bits[j]
    return out


def quantize_row(x_bits, offsets, ts, rounding=0, seed=0, offset=0):
    """(codes, scales, owned): owned tells the rows that an expert has."""
    codes, scales = quantize.quantize_blockscale(x_bits, ts, rounding, seed, offset, 0)
    owned = np.zeros(x_bits.shape[0], dtype=bool)
    for b, n, _, _ in spans(offsets):
        owned[b:b + n] = True
    return codes, scales, owned


def quantize_col(x_bits, offsets, ts, rounding=0, seed=0, offset=0):
    """(codes, scales, written): written tells the columns (in blocks of 16) that are some expert's."""
    rows, cols = x_bits.shape
    wide = np.zeros((rows_padded(rows, len(offsets) - 1), cols), dtype=np.uint16)
    written = np.zeros(wide.shape[0] // 16, dtype=bool)
    for b, n, p, np_ in spans(offsets):
        wide[p:p + n] = x_bits[b:b + n]
        written[p // 16:(p + np_) // 16] = True
    codes, scales = quantize.quantize_blockscale(wide, ts, rounding, seed, offset, 1)
    return codes, scales, written


def amax(x_bits, offsets):
    """max |x| over the experts' rows (a NaN propagates)."""
    rows = [x_bits[b:b + n] for b, n, _, _ in spans(offsets)]
    return quantize.tensor_amax(np.concatenate(rows))


def gemm_rows(a, ts_a, b_codes, b_scales, ts_b, offsets):
    """fprop and dgrad: (C, bound, owned) with NaN-free zeros in the rows of no expert."""
    rows, N = a[0].shape[0], b_codes.shape[1]
    c, bound, owned = np.zeros((rows, N)), np.zeros((rows, N)), np.zeros(rows, dtype=bool)
    for g, (b, n, _, _) in enumerate(spans(offsets)):
        c[b:b + n], bound[b:b + n] = gemm.gemm_nt(a[0][b:b + n], a[1][b:b + n], ts_a, b_codes[g], b_scales[g], ts_b[g])
        owned[b:b + n] = True
    return c, bound, owned


def gemm_wgrad(a, ts_a, b, ts_b, offsets):
    """(C [experts][M][N], bound) over each expert's columns of the transposed operands."""
    c, bound = [], []
    for _, _, p, n in spans(offsets):
        part = [(q[0][:, p // 2:(p + n) // 2], q[1][:, p // 16:(p + n) // 16]) for q in (a, b)]
        v = gemm.gemm_nt(*part[0], ts_a, *part[1], ts_b)
        c.append(v[0])
        bound.append(v[1])
    return np.stack(c), np.stack(bound)


def weight_only(x_bits, w_codes, w_scales, w_ts, offsets):
    """(C, bound, owned): bf16 rows times the dequantized weights of their expert, in fp64."""
    x = formats.bf16_to_f32(x_bits).astype(np.float64)
    rows, N = x.shape[0], w_codes.shape[1]
    c, bound, owned = np.zeros((rows, N)), np.zeros((rows, N)), np.zeros(rows, dtype=bool)
    for g, (b, n, _, _) in enumerate(spans(offsets)):
        w = quantize.dequantize_unscaled(w_codes[g], w_scales[g])
        ts = float(np.float32(w_ts[g]))
        with np.errstate(invalid="ignore", over="ignore"):
            c[b:b + n] = ts * (x[b:b + n] @ w.T)
            bound[b:b + n] = abs(ts) * (np.abs(x[b:b + n]) @ np.abs(w).T)
        owned[b:b + n] = True
    return c, bound, owned
