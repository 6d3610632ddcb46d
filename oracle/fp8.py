"""8-bit block-128 quantization and its GEMM (oracle side).

TEST INFRASTRUCTURE: see oracle/__init__.py for who may use this module.

Formats: OCP FP8 E4M3 (bias 7, largest 448) and E5M2 (bias 15, largest finite
57344).  Reading for the arithmetic (fp32, one IEEE rounding per operation):
  1. blocks of 128 along the columns of the output orientation, the last one
     short where the columns are no multiple of 128; or aligned 128 x 128 tiles;
  2. amax = max |x| over the block;
  3. fp32 scale: s = max(fp32(amax / F), 2^-126); E8M0 scale: s = the least
     power of two >= amax / F, at least 2^-127, stored as its exponent + 127;
  4. code = the format's value nearest to fp32(x * fp32(1 / s)), ties to even
     (never beyond F: amax * (1 / s) is F to within an fp32 rounding);
  5. a block whose amax is not finite: scale NaN (E8M0 0xFF), codes 0.
Codes are padded with zeros to a multiple of 128 columns; scales are laid out
block index first.
"""

import numpy as np

from . import formats

E4M3 = 0
E5M2 = 1
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
_BITS = {E4M3: (3, 7), E5M2: (2, 15)}  # mantissa bits, exponent bias


def decode(codes, fmt):
    """float64 values of 8-bit codes."""
    m, bias = _BITS[fmt]
    c = np.asarray(codes, dtype=np.int64)
    e, f = (c & 0x7F) >> m, c & ((1 << m) - 1)
    v = np.where(e == 0, np.ldexp(f.astype(np.float64), 1 - bias - m),
                 np.ldexp(1.0 + f / (1 << m), e - bias))
    if fmt == E4M3:
        v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(e == 31, np.where(f == 0, np.inf, np.nan), v)
    return np.where(c & 0x80, -v, v)


def encode(v, fmt):
    """Codes of the nearest values (ties to even) of finite v, |v| below the
    point half a step past the largest value; the sign of zeros is kept."""
    m, bias = _BITS[fmt]
    a = np.abs(np.asarray(v, dtype=np.float64))
    _, e = np.frexp(a)                       # a = f 2^e, f in [0.5, 1)
    e = np.where(a == 0, 1 - bias, np.maximum(e - 1, 1 - bias))  # exponent of the step's binade
    q = np.rint(np.ldexp(a, m - e)).astype(np.int64)  # in units of 2^(e - m)
    code = q + ((e + bias - 1) << m)         # a carry runs into the exponent
    return (code | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def block_scale(amax, fmt, e8m0):
    """(stored scale, fp32 reciprocal) of block maxima (float32)."""
    amax = np.asarray(amax, dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        q = (amax / np.float32(LARGEST[fmt])).astype(np.float32)
    finite = np.isfinite(amax)
    if e8m0:
        f, e = np.frexp(np.where(finite, q, np.float32(1.0)).astype(np.float64))
        e = np.where(f == 0.5, e - 1, e)
        e = np.maximum(np.where(q == 0, -127, e), -127)
        r = np.ldexp(np.float64(1.0), -e).astype(np.float32)
        return np.where(finite, e + 127, 0xFF).astype(np.uint8), r
    s = np.where(finite, np.maximum(q, np.float32(2.0 ** -126)), np.float32(np.nan)).astype(np.float32)
    return s, (np.float32(1.0) / s).astype(np.float32)


def quantize(x_bits, fmt, e8m0=False, tile=False, orientation=0):
    """(codes [R][Cp], scales [Cp / 128][R or ceil(R / 128)]) of the bf16 matrix
    (orientation 1: of its transpose)."""
    x = formats.bf16_to_f32(np.asarray(x_bits, dtype=np.uint16))
    x = x if orientation == 0 else x.T
    R, C = x.shape
    nb, g = (C + 127) // 128, 128 if tile else 1
    ng = (R + g - 1) // g
    w = np.zeros((ng * g, nb * 128), dtype=np.float32)
    w[:R, :C] = x
    w = w.reshape(ng, g, nb, 128)
    amax = np.max(np.abs(w), axis=(1, 3))    # NaN propagates
    stored, r = block_scale(amax, fmt, e8m0)
    ok = np.isfinite(amax)[:, None, :, None]
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        v = (np.where(ok, w, np.float32(0.0)) * np.where(np.isfinite(r), r, np.float32(1.0))[:, None, :, None]).astype(np.float32)
    codes = np.where(ok, encode(v, fmt), 0).astype(np.uint8)
    return codes.reshape(ng * g, nb * 128)[:R], np.ascontiguousarray(stored.T)


def scale_values(scales):
    """float64 values of fp32 or E8M0 scales."""
    if scales.dtype == np.uint8:
        return np.where(scales == 0xFF, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return scales.astype(np.float64)


def operand(codes, scales, fmt, tile):
    """float64 values [R][Cp] of a quantized operand."""
    R, nb = codes.shape[0], codes.shape[1] // 128
    s = scale_values(scales)                  # [nb][rows or tiles]
    s = s[:, np.arange(R) // 128] if tile else s
    return (decode(codes, fmt).reshape(R, nb, 128) * s.T[:, :, None]).reshape(R, nb * 128)


def gemm_nt(a, b):
    """(A B^T, |A| |B|^T) in fp64 of two operands' values."""
    return a @ b.T, np.abs(a) @ np.abs(b).T
