// 8-bit quantizer: bf16 -> E4M3 / E5M2 codes with one scale per block of 128
// (1 x 128 along each output's contraction axis, or 128 x 128 tiles), the
// row-wise and the transposed operand from one read of the input.  Arithmetic
// and layouts: include/ue5m3fp4_layer.h.
//
// Work split.  A 256-thread workgroup owns a 128 x 128 tile: every block of
// either orientation lies in one tile, and a tile's codes are whole 128-byte
// lines of both outputs.  Thread t loads 16-byte unit t % 16 (8 columns) of
// tile rows t / 16 + 16 k, k < 8; what lies outside the tensor is zero, which
// changes no amax and gives the codes' zero padding.
//  - Row-wise pass, from registers: a block spans the 16 lanes of a DPP row.
//    The amaxes of the 8 rows meet there (two rows per packed 16-bit max),
//    lane u computes the scale of row u % 8 and broadcasts it.
//  - Transposed pass, through LDS (XOR-swizzled, conflict-free): a lane quad
//    owns a column pair, each lane 16 rows of either half, so that the quad's
//    stores run over 64 contiguous bytes.
//  - Tile order: bands of 4 tile rows, walked column by column: the tiles in
//    flight then write runs of 512 bytes of each column of the transposed codes.
//    Row by row the 8192 x 16384 case below takes 115 us, in bands of 16 rows
//    122; a contiguous range per XCD loses 5-10 % (the outputs are whole lines,
//    so no two tiles share one that an L2 would have to merge).
//  - Cache policy: x is read once and the row-wise codes leave as whole lines per
//    store, both non-temporal; the transposed codes leave as two stores of half a
//    line and have to meet in L2 (non-temporal: 120 instead of 115 us).
//
// Bound: HBM.  Both outputs, inputs and outputs rotated past the 256 MB cache:
// 8192 x 4096 28 us (4.9 TB/s), 8192 x 16384 110 us (4.9), 16384 x 4096 in tiles
// 47 us (5.7); a plain copy of these sizes runs at 5.2 to 5.9.  Without the
// divisions, or without the scale stores, the times are the same within 2 %.
#include "../formats.hpp"
#include "layer.hpp"

namespace ue5m3fp4 {

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr uint32_t kBand = 4;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;  // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kRowRor = 0x120;                     // + n: rotate the 16 lanes of a row by n
constexpr int kRowBcast = 0x150;                   // + n: lane n of the row, to all of it

struct Scale {
    float s;        // the fp32 scale, or
    uint32_t byte;  // the E8M0 scale
    float r;        // 1 / scale
    uint32_t mask;  // all ones; 0 for a block that is not finite (zero codes)
};

// Scale of a block with amax bits `bits` (bf16 magnitude).
template <bool E5M2, bool E8M0>
__device__ __forceinline__ Scale block_scale(uint32_t bits) {
    const bool finite = bits < 0x7F80u;
    const float q = __uint_as_float(bits << 16) / (E5M2 ? 57344.0f : 448.0f);
    Scale o;
    o.mask = finite ? 0xFFFFFFFFu : 0u;
    if (E8M0) {
        const uint32_t b = __float_as_uint(q);
        const uint32_t e = b <= 0x00400000u ? 0u : (b >> 23) + ((b & 0x7FFFFFu) != 0u);  // 2^(e - 127) >= q
        o.byte = finite ? e : 0xFFu;
        o.r = __uint_as_float((254u - min(e, 253u)) << 23);
        o.s = 0.0f;
    } else {
        o.s = finite ? fmaxf(q, 0x1p-126f) : __uint_as_float(0x7FC00000u);
        o.r = 1.0f / o.s;
        o.byte = 0u;
    }
    return o;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    int w;
    if constexpr (E5M2) {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    }
    return (uint32_t)w;
}

template <bool E8M0>
__device__ __forceinline__ void put_scale(void* base, int64_t at, const Scale& o) {
    if constexpr (E8M0) ((uint8_t*)base)[at] = (uint8_t)o.byte;
    else ((float*)base)[at] = o.s;
}

// 8 columns from c0 of row r, zero outside the tensor.  vec: rows are 16-byte
// aligned.
__device__ __forceinline__ u32x4 load_unit(const QuantizeFp8Args& a, int64_t r, int64_t c0, bool vec) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (r >= a.rows || c0 >= a.cols) return w;
    const uint16_t* p = a.x + r * a.ld + c0;
    if (vec && c0 + 8 <= a.cols) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (c0 + e < a.cols) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    return w;
}

template <bool E5M2, bool E8M0, bool TILE, bool ROW, bool COL>
__global__ __launch_bounds__(kThreads) void quantize_fp8_kernel(QuantizeFp8Args a) {
    __shared__ __align__(16) uint8_t tile[COL ? kTile * kTile * 2 : 16];
    __shared__ uint32_t wave_max[kThreads / 64];
    const int t = threadIdx.x, u = t & 15, rb = t >> 4;
    const uint32_t tiles_c = (uint32_t)((a.cols + kTile - 1) / kTile);
    const uint32_t tiles_r = (uint32_t)((a.rows + kTile - 1) / kTile);
    const uint32_t id = blockIdx.x + (uint32_t)a.first;
    const uint32_t band = id / (kBand * tiles_c), rem = id - band * kBand * tiles_c;
    const uint32_t height = min(kBand, tiles_r - kBand * band);
    const int64_t tr = kBand * band + rem % height, tc = rem / height;
    const int64_t R0 = tr * kTile, C0 = tc * kTile, c0 = C0 + 8 * u;
    const int64_t Cp = (int64_t)tiles_c * kTile, Rp = (int64_t)tiles_r * kTile;

    u32x4 w[8];
    if (R0 + kTile <= a.rows && C0 + kTile <= a.cols && a.ld % 8 == 0) {
        const uint16_t* src = a.x + (R0 + rb) * a.ld + c0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + (int64_t)(16 * k) * a.ld));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = load_unit(a, R0 + rb + 16 * k, c0, a.ld % 8 == 0);
    }

    // amax of the 8 rows' units, two rows per word (rows 2m and 2m + 1)
    uint32_t hm[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        uint32_t x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 v = w[2 * m + i];
            const uint32_t y = pk_max(pk_max(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), pk_max(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
            x[i] = max(y & 0xFFFFu, y >> 16);
        }
        hm[m] = x[0] | (x[1] << 16);
    }

    Scale ts;  // TILE: the tile's scale
    if (TILE) {
        uint32_t m = pk_max(pk_max(hm[0], hm[1]), pk_max(hm[2], hm[3]));
        m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s));
        if ((t & 63) == 0) wave_max[t >> 6] = m;
    }
    if (COL) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int row = rb + 16 * k;
            *reinterpret_cast<u32x4*>(tile + row * (kTile * 2) + ((u ^ (((row >> 4) & 3) << 2)) << 4)) = w[k];
        }
    }
    if (TILE || COL) __syncthreads();
    if (TILE) {
        ts = block_scale<E5M2, E8M0>(max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3])));
        if (t == 0) {
            if (ROW) put_scale<E8M0>(a.row_scales, tc * tiles_r + tr, ts);
            if (COL) put_scale<E8M0>(a.col_scales, tr * (int64_t)tiles_c + tc, ts);
        }
    }

    if (ROW) {
        float r[8];
        uint32_t mask[8];
        if (TILE) {
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = ts.r, mask[k] = ts.mask;
        } else {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                hm[m] = pk_max(hm[m], dpp<kRowRor + 8>(hm[m]));
                hm[m] = pk_max(hm[m], dpp<kRowRor + 4>(hm[m]));
                hm[m] = pk_max(hm[m], dpp<kRowRor + 2>(hm[m]));
                hm[m] = pk_max(hm[m], dpp<kRowRor + 1>(hm[m]));
            }
            const uint32_t pair = (u & 4) ? ((u & 2) ? hm[3] : hm[2]) : ((u & 2) ? hm[1] : hm[0]);
            const Scale mine = block_scale<E5M2, E8M0>((u & 1) ? pair >> 16 : pair & 0xFFFFu);
            if (u < 8 && R0 + rb + 16 * u < a.rows)
                put_scale<E8M0>(a.row_scales, tc * a.rows + R0 + rb + 16 * u, mine);
            const uint32_t rbits = __float_as_uint(mine.r);
#define UE5M3FP4_BCAST(k)                                  \
    r[k] = __uint_as_float(dpp<kRowBcast + k>(rbits));     \
    mask[k] = dpp<kRowBcast + k>(mine.mask);
            UE5M3FP4_BCAST(0) UE5M3FP4_BCAST(1) UE5M3FP4_BCAST(2) UE5M3FP4_BCAST(3)
            UE5M3FP4_BCAST(4) UE5M3FP4_BCAST(5) UE5M3FP4_BCAST(6) UE5M3FP4_BCAST(7)
#undef UE5M3FP4_BCAST
        }
        uint8_t* dst = a.row_codes + (R0 + rb) * Cp + c0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            u32x2 o;
            o.x = encode4<E5M2>(bf16_lo(w[k].x) * r[k], bf16_hi(w[k].x) * r[k], bf16_lo(w[k].y) * r[k], bf16_hi(w[k].y) * r[k]);
            o.y = encode4<E5M2>(bf16_lo(w[k].z) * r[k], bf16_hi(w[k].z) * r[k], bf16_lo(w[k].w) * r[k], bf16_hi(w[k].w) * r[k]);
            o.x &= mask[k];
            o.y &= mask[k];
            if (R0 + rb + 16 * k < a.rows)
                __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(dst + (int64_t)(16 * k) * Cp));
        }
    }

    if (COL) {
        const int seg = t & 3, cp = t >> 2;  // rows 16 seg .. + 15 of either half, column pair
        const int64_t ca = C0 + 2 * cp;
        uint32_t v[32];
        const uint8_t* src = tile + seg * 16 * (kTile * 2) + (((cp >> 2) ^ (seg << 2)) << 4) + 4 * (cp & 3);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = *reinterpret_cast<const uint32_t*>(src + (i < 16 ? i : i + 48) * (kTile * 2));
        float ra, rb2;
        uint32_t ma, mb;
        if (TILE) {
            ra = rb2 = ts.r;
            ma = mb = ts.mask;
        } else {
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i) m = pk_max(m, v[i] & 0x7FFF7FFFu);
            m = pk_max(m, dpp<kQuadXor1>(m));
            m = pk_max(m, dpp<kQuadXor2>(m));
            // even lanes of the quad take column a, odd ones column b
            const Scale mine = block_scale<E5M2, E8M0>((seg & 1) ? m >> 16 : m & 0xFFFFu);
            if (seg < 2 && ca + seg < a.cols) put_scale<E8M0>(a.col_scales, tr * a.cols + ca + seg, mine);
            const float other = __uint_as_float(dpp<kQuadXor1>(__float_as_uint(mine.r)));
            const uint32_t omask = dpp<kQuadXor1>(mine.mask);
            ra = (seg & 1) ? other : mine.r;
            rb2 = (seg & 1) ? mine.r : other;
            ma = (seg & 1) ? omask : mine.mask;
            mb = (seg & 1) ? mine.mask : omask;
        }
        uint8_t* dst = a.col_codes + ca * Rp + R0 + 16 * seg;
        u32x4 o[2];
        if (ca < a.cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i >> 2][i & 3] = ma & encode4<E5M2>(bf16_lo(v[4 * i]) * ra, bf16_lo(v[4 * i + 1]) * ra,
                                                      bf16_lo(v[4 * i + 2]) * ra, bf16_lo(v[4 * i + 3]) * ra);
            *reinterpret_cast<u32x4*>(dst) = o[0];
            *reinterpret_cast<u32x4*>(dst + 64) = o[1];
        }
        if (ca + 1 < a.cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i >> 2][i & 3] = mb & encode4<E5M2>(bf16_hi(v[4 * i]) * rb2, bf16_hi(v[4 * i + 1]) * rb2,
                                                      bf16_hi(v[4 * i + 2]) * rb2, bf16_hi(v[4 * i + 3]) * rb2);
            *reinterpret_cast<u32x4*>(dst + Rp) = o[0];
            *reinterpret_cast<u32x4*>(dst + Rp + 64) = o[1];
        }
    }
}

template <bool E5M2, bool E8M0, bool TILE, bool ROW, bool COL>
void launch_tiles(const QuantizeFp8Args& a, hipStream_t stream) {
    in_launches(((a.rows + kTile - 1) / kTile) * ((a.cols + kTile - 1) / kTile), kThreads, [&](int64_t first, dim3 grid) {
        QuantizeFp8Args part = a;
        part.first = first;
        hipLaunchKernelGGL((quantize_fp8_kernel<E5M2, E8M0, TILE, ROW, COL>), grid, dim3(kThreads), 0, stream, part);
    });
}

template <bool E5M2, bool E8M0, bool TILE>
void launch_outputs(const QuantizeFp8Args& a, hipStream_t stream) {
    if (a.row_codes && a.col_codes) launch_tiles<E5M2, E8M0, TILE, true, true>(a, stream);
    else if (a.row_codes) launch_tiles<E5M2, E8M0, TILE, true, false>(a, stream);
    else launch_tiles<E5M2, E8M0, TILE, false, true>(a, stream);
}

template <bool E5M2, bool E8M0>
void launch_tile(const QuantizeFp8Args& a, hipStream_t stream) {
    a.tile ? launch_outputs<E5M2, E8M0, true>(a, stream) : launch_outputs<E5M2, E8M0, false>(a, stream);
}

}  // namespace

void launch_quantize_fp8(const QuantizeFp8Args& a, hipStream_t stream) {
    if (a.e5m2) a.e8m0 ? launch_tile<true, true>(a, stream) : launch_tile<true, false>(a, stream);
    else a.e8m0 ? launch_tile<false, true>(a, stream) : launch_tile<false, false>(a, stream);
}

}  // namespace ue5m3fp4
