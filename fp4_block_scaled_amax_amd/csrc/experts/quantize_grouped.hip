// Block-16 E2M1/UE5M3 quantizer of rows grouped by expert (gfx950): row-wise
// operand, grouped transposed operand and amax from one read of each row,
// gathered by an index where there is one.
//
// Method: "UE5M3 FP4 Block Scaling for Stable Language Model Pretraining"
// (arXiv 2609.02846), abstract; the arithmetic per block is quant_block.hpp's.
//
// Work decomposition.  A 256-thread workgroup owns TR rows x 256 columns of the
// rows_padded x cols matrix that the transposed operand is blocked along (each
// expert's rows from a multiple of 128 on), so a tile has rows of one expert
// and both outputs come from one read.  Which expert: the last whose first
// padded row is not behind the tile's, found by ballots in each wave, among 64
// ranges of experts and then in the range, without a scan or a second kernel (1024
// experts, 4096 x 1024, mostly padding: 62 us, 64 experts after another 85).  Tiles in
// the gaps end there.  Rows of a tile behind the expert's last are zeros, which
// quantize to the operand's padding.
//
// Thread t loads 16-byte unit t % 32 (8 columns) of tile rows t / 32 + 8k, all
// loads issued back to back; the row-wise pass quantizes from registers (a lane
// pair shares a block), the transposed pass from an XOR-swizzled LDS tile, one
// 16-row block of two neighbouring columns per lane.
#include "../formats.hpp"
#include "../quant_block.hpp"
#include "experts.hpp"

namespace ue5m3fp4 {

namespace {

// Tile height: 64 with the transposed output (32-byte runs of its codes), else
// 32 (more resident workgroups hide more of the loads' latency).
template <int TR>
struct Shape {
    static constexpr int kRowsPerThread = TR / 8;          // tile rows t / 32 + 8k
    static constexpr int kRowBlocks = TR / 16;             // 16-row blocks per column
    static constexpr int kPairsPerWave = 64 / kRowBlocks;  // column pairs per wave and pass
    static constexpr int kColPasses = 128 / (4 * kPairsPerWave);
    static constexpr int kBand = 256 / TR;                 // tiles that share lines of the transposed output
    static_assert(TR == 32 || TR == 64, "a tile is inside a group's 128 rows");
};
constexpr int kTileCols = 256;
constexpr int kThreads = 256;
constexpr int kLdsRowBytes = kTileCols * 2;  // one bf16 tile row

// LDS position of 16-byte unit u of tile row `row`: the unit is XORed with the
// row's 16-row block, so that the transposed pass (lanes over row blocks and
// column pairs) reads 64 distinct banks.
template <int TR>
__device__ __forceinline__ int lds_offset(int row, int u) {
    constexpr int kRowBlocks = Shape<TR>::kRowBlocks;
    return row * kLdsRowBytes + ((u ^ (((row >> 4) & (kRowBlocks - 1)) * (16 / kRowBlocks))) << 4);
}

// Workgroup number -> tile: each XCD takes a contiguous range of an order that
// runs down bands of 256 rows column by column, so that tiles which share lines of
// the transposed codes meet in one L2.  The numbers fit 32 bits: cols * rows_padded
// < 2^40, and a tile has 32 x 256 elements, or at least 32 rows.
template <int TR>
__device__ __forceinline__ void tile_of(uint32_t j, uint32_t tiles_r, uint32_t tiles_c, int64_t& R0, int64_t& C0) {
    constexpr uint32_t kBand = Shape<TR>::kBand;
    const uint32_t per_xcd = tiles_r * tiles_c / 8;
    if (j < per_xcd * 8) j = (j % 8) * per_xcd + j / 8;  // the tail keeps its number
    const uint32_t band = j / (kBand * tiles_c), rem = j - band * kBand * tiles_c;
    const uint32_t h = min(kBand, tiles_r - kBand * band), column = rem / h;
    C0 = (int64_t)column * kTileCols;
    R0 = (int64_t)(kBand * band + rem - column * h) * TR;
}

// block_scale, which leaves tiny blocks under K < 1 to the general path, for a tile
// whose last rows may be zeros: a zero block has code 0 and r = 0 there like any
// other that flushes.  (Left to the general path, the last tiles of 16 experts' rows
// made a call on 16384 x 4096 take 69 us instead of 48.)
__device__ __forceinline__ BlockScale scale_of(uint32_t amax16, const Ctx& ctx, const float* rlut, bool& ok) {
    bool fast = ctx.fastK;
    const BlockScale b = block_scale(amax16, ctx, rlut, fast);
    ok = ok & (fast | ((amax16 == 0u) & ctx.fastK));
    return b;
}

// Largest magnitude (bf16 bits) of the workgroup folded into *amax: one atomic
// per workgroup, none where the running value is as large (it only grows).
__device__ __forceinline__ void amax_commit(uint32_t m, float* amax) {
    __shared__ uint32_t wave_max[kThreads / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        m = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
        unsigned int* dst = reinterpret_cast<unsigned int*>(amax);
        if (m != 0u && (m << 16) > __hip_atomic_load(dst, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT))
            atomicMax(dst, m << 16);
    }
}

// W32: every call number of the stochastic rounding is below 2^32, so the counter's
// second word is 0 and the half of the first rounds that depends on it is the same in
// all lanes.  ONCE: no index, so each row is read once, past the caches.
template <int TR, bool ROW, bool COL, bool SR, bool W32, bool ONCE>
__global__ __launch_bounds__(kThreads) void quantize_grouped_kernel(QuantizeGroupedArgs a, int64_t first) {
    using S = Shape<TR>;
    constexpr int kRowsPerThread = S::kRowsPerThread, kRowBlocks = S::kRowBlocks, kPairsPerWave = S::kPairsPerWave;
    __shared__ __align__(16) uint8_t tile[COL ? TR * kLdsRowBytes : 16];
    __shared__ float rlut[(ROW || COL) ? 256 : 1];
    const int t = threadIdx.x, lane = t & 63;
    const int64_t padded = 128 * ((a.rows + 127) / 128 + a.experts);
    int64_t R0, C0;
    tile_of<TR>((uint32_t)first + blockIdx.x, (uint32_t)(padded / TR), (uint32_t)((a.cols + kTileCols - 1) / kTileCols), R0, C0);

    // ---- the tile's expert, and the grouped rows [row0, end) it has here
    const float ts = (ROW || COL) ? *a.tensor_scale : 0.0f;
    int low = 0, candidates = a.experts;
    while (candidates > 64) {  // which of 64 ranges of experts
        const int step = (candidates + 63) / 64, e = low + lane * step;
        const bool before = lane * step < candidates && padded_begin(group_rows(a.offsets, e, (int)a.rows).begin, e) <= R0;
        const int begun = (int)__popcll(__ballot(before)), last = begun > 0 ? begun - 1 : 0;
        candidates = min(step, candidates - last * step);
        low += last * step;
    }
    GroupRows own{0, 0};
    bool before = false;
    if (lane < candidates) {
        own = group_rows(a.offsets, low + lane, (int)a.rows);
        before = padded_begin(own.begin, low + lane) <= R0;
    }
    const int last = __popcll(__ballot(before)) - 1;
    if (last < 0) return;  // before the first expert's rows
    const int g = low + last;
    own.begin = __shfl(own.begin, last);
    own.end = __shfl(own.end, last);
    const int64_t rel = R0 - padded_begin(own.begin, g);
    const int64_t end = own.end, row0 = own.begin + rel;
    // behind the expert's padding (or, for the row-wise output alone, its rows);
    // before its first row only where the offsets decrease
    if (rel < 0 || (COL ? rel >= (end - own.begin + 127) / 128 * 128 : row0 >= end)) return;

    // padding alone: zeros, unless the tensor scale makes a zero block NaN (0 / 0)
    if (COL && row0 >= end && 6.0f * ts != 0.0f && ts == ts) {
        const int column = t;
        if (C0 + column < a.cols) {
#pragma unroll
            for (int k = 0; k < TR / 32; ++k)
                *reinterpret_cast<u32x4*>(a.col_codes + (C0 + column) * (padded / 2) + R0 / 2 + 16 * k) = u32x4{0u, 0u, 0u, 0u};
            *reinterpret_cast<uint32_t*>(a.col_scales + (C0 + column) * (padded / 16) + R0 / 16) = 0u;
        }
        return;
    }

    // ---- loads: 16-byte unit u of tile rows rbase + 8k; rows that are not the
    // expert's, or whose index is out of range, are zeros.  Addresses are clamped
    // into x, so every load is unconditional.
    const int u = t & 31, rbase = t >> 5;
    const int64_t c0 = C0 + 8 * u;
    const bool col_ok = c0 < a.cols, interior = row0 + TR <= end && C0 + kTileCols <= a.cols;
    const uint16_t* src = a.x + (col_ok ? c0 : a.cols - 8);
    u32x4 w[kRowsPerThread];
    uint32_t zero = 0u;  // bit k: row k is not there
    if (ONCE) {
        if (interior) {  // one base address, then a stride common to the launch
            src += (row0 + rbase) * a.ld;
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k)
                w[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + (int64_t)(8 * k) * a.ld));
        } else {
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k) {
                const int64_t r = row0 + rbase + 8 * k;
                if (r >= end) zero |= 1u << k;
                w[k] = *reinterpret_cast<const u32x4*>(src + min(r, a.rows - 1) * a.ld);
            }
        }
    } else {
        int32_t from[kRowsPerThread];
        const int32_t* index = a.index + row0 + rbase;
#pragma unroll
        for (int k = 0; k < kRowsPerThread; ++k) from[k] = index[interior ? 8 * k : min((int64_t)(8 * k), a.rows - 1 - row0 - rbase)];
#pragma unroll
        for (int k = 0; k < kRowsPerThread; ++k) {
            if ((uint32_t)from[k] >= (uint32_t)a.x_rows || (!interior && row0 + rbase + 8 * k >= end)) {
                zero |= 1u << k;
                from[k] = 0;
            }
        }
        if (a.x_rows > 0) {
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k) w[k] = *reinterpret_cast<const u32x4*>(src + (uint32_t)from[k] * a.ld);
        }
    }
    if (__any(zero)) {
#pragma unroll
        for (int k = 0; k < kRowsPerThread; ++k)
            if ((zero >> k) & 1u) w[k] = u32x4{0u, 0u, 0u, 0u};
    }

    Ctx ctx{0.0f, 0.0f, 0.0f, false, false};
    if (ROW || COL) {
        ctx = make_ctx(ts);
        rlut[t] = rcp_entry<SR>((uint32_t)t, ctx.ts);
    }

    // ---- half-block amax (bf16 magnitude bits; NaN sorts above Inf)
    uint32_t hmax[kRowsPerThread];
    uint32_t tmax = 0u;
#pragma unroll
    for (int k = 0; k < kRowsPerThread; ++k) {
        hmax[k] = max_abs8(w[k]);
        tmax = max(tmax, col_ok ? hmax[k] : 0u);
    }
    if (COL) {
#pragma unroll
        for (int k = 0; k < kRowsPerThread; ++k)
            *reinterpret_cast<u32x4*>(tile + lds_offset<TR>(rbase + 8 * k, u)) = w[k];
    }
    if (ROW || COL) __syncthreads();  // reciprocal table (and tile) visible

    // ---- row-wise output: the lane pair (t, t ^ 1) shares each block; lane
    // parity p computes the scales of rows k = 2m + p and the pair swaps them
    if (ROW) {
        const uint32_t p = t & 1;
        uint32_t code[kRowsPerThread];
        float rr[kRowsPerThread];
        bool ok = ctx.fastK;
#pragma unroll
        for (int m = 0; m < kRowsPerThread / 2; ++m) {
            const uint32_t mine = p ? hmax[2 * m + 1] : hmax[2 * m];
            const uint32_t other = p ? hmax[2 * m] : hmax[2 * m + 1];
            const BlockScale b = scale_of(max(mine, swap_pair(other)), ctx, rlut, ok);
            const uint32_t pc = swap_pair(b.code);
            const float pr = __uint_as_float(swap_pair(__float_as_uint(b.r)));
            code[2 * m] = p ? pc : b.code;
            rr[2 * m] = p ? pr : b.r;
            code[2 * m + 1] = p ? b.code : pc;
            rr[2 * m + 1] = p ? b.r : pr;
        }
        const uint32_t ok_bit = ok ? 1u : 0u;
        const bool pair_ok = (ok_bit & swap_pair(ok_bit)) != 0u;  // one path for both lanes of a pair
        uint32_t packed[kRowsPerThread];
        auto words = [&](int k) {
            const uint64_t n = ((uint64_t)(row0 + rbase + 8 * k) * (uint64_t)a.cols + (uint64_t)c0) >> 3;
            return W32 ? sr_words32((uint32_t)n, a.offset, 0u, a.seed) : sr_words(n, a.offset, 0u, a.seed);
        };
        if (__builtin_expect(pair_ok, 1)) {
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k) {
                float v[8];
                unpack8(w[k], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * rr[k];
                U32x4 rnd;
                if (SR) rnd = words(k);
                packed[k] = encode8<SR>(v, rnd);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k) {
                const BlockScale b = block_scale_general(max(hmax[k], swap_pair(hmax[k])), ctx.ts, ctx.K);
                U32x4 rnd;
                if (SR) rnd = words(k);
                packed[k] = encode8_general<SR>(w[k], b.code, b.r, rnd);
                code[k] = b.code;
            }
        }
        uint8_t* pc = a.row_codes + (row0 + rbase) * (a.cols / 2) + c0 / 2;
        uint8_t* ps = a.row_scales + (row0 + rbase) * (a.cols / 16) + c0 / 16;
        const int64_t cstep = 8 * (a.cols / 2), sstep = 8 * (a.cols / 16);
        if (interior) {  // both lanes of a pair store the block's scale byte
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k) {
                __builtin_nontemporal_store(packed[k], reinterpret_cast<uint32_t*>(pc + k * cstep));
                ps[k * sstep] = (uint8_t)code[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < kRowsPerThread; ++k) {
                if (col_ok && row0 + rbase + 8 * k < end) {
                    *reinterpret_cast<uint32_t*>(pc + k * cstep) = packed[k];
                    if (p == 0) ps[k * sstep] = (uint8_t)code[k];
                }
            }
        }
    }

    // ---- transposed output: lane (rb, cp) of wave wv quantizes columns 2j, 2j +
    // 1 over tile rows 16 rb .. 16 rb + 15, one block per column
    if (COL) {
        const int wv = t >> 6, rb = lane % kRowBlocks, cp = lane / kRowBlocks;
        const int64_t r0 = R0 + 16 * rb;  // padded row of the block
#pragma unroll 1
        for (int pass = 0; pass < S::kColPasses; ++pass) {
            const int j = kPairsPerWave * (wv + 4 * pass) + cp;
            const int64_t ca = C0 + 2 * j;
            uint32_t cw[16];
            const uint8_t* from_lds = tile + lds_offset<TR>(16 * rb, j >> 2) + 4 * (j & 3);
#pragma unroll
            for (int i = 0; i < 16; ++i) cw[i] = *reinterpret_cast<const uint32_t*>(from_lds + i * kLdsRowBytes);
            uint32_t m2 = 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) m2 = pk_max_u16(m2, cw[i] & 0x7FFF7FFFu);
            bool ok = ctx.fastK;
            BlockScale ba = scale_of(m2 & 0xFFFFu, ctx, rlut, ok);
            BlockScale bb = scale_of(m2 >> 16, ctx, rlut, ok);
            U32x4 rnd[4];
            if (SR) {
                const uint64_t na = ((uint64_t)ca * (uint64_t)padded + (uint64_t)r0) >> 3;
                const uint64_t nb = na + (uint64_t)(padded >> 3);
                auto words = [&](uint64_t n) {
                    return W32 ? sr_words32((uint32_t)n, a.offset, 1u, a.seed) : sr_words(n, a.offset, 1u, a.seed);
                };
                rnd[0] = words(na);
                rnd[1] = words(na + 1u);
                rnd[2] = words(nb);
                rnd[3] = words(nb + 1u);
            }
            uint32_t pa[2], pb[2];
            if (__builtin_expect(ok, 1)) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float va[8], vb[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        va[i] = bf16_lo(cw[8 * hh + i]) * ba.r;
                        vb[i] = bf16_hi(cw[8 * hh + i]) * bb.r;
                    }
                    pa[hh] = encode8<SR>(va, rnd[hh]);
                    pb[hh] = encode8<SR>(vb, rnd[2 + hh]);
                }
            } else {
                ba = block_scale_general(m2 & 0xFFFFu, ctx.ts, ctx.K);
                bb = block_scale_general(m2 >> 16, ctx.ts, ctx.K);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t la[4], lb[4];  // words of one column, two rows each
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w0 = cw[8 * hh + 2 * i], w1 = cw[8 * hh + 2 * i + 1];
                        la[i] = (w0 & 0xFFFFu) | (w1 << 16);
                        lb[i] = (w0 >> 16) | (w1 & 0xFFFF0000u);
                    }
                    pa[hh] = encode8_general<SR>(u32x4{la[0], la[1], la[2], la[3]}, ba.code, ba.r, rnd[hh]);
                    pb[hh] = encode8_general<SR>(u32x4{lb[0], lb[1], lb[2], lb[3]}, bb.code, bb.r, rnd[2 + hh]);
                }
            }
            if (interior || ca < a.cols) {  // columns come in pairs: cols % 16 == 0
                *reinterpret_cast<u32x2*>(a.col_codes + ca * (padded / 2) + r0 / 2) = u32x2{pa[0], pa[1]};
                *reinterpret_cast<u32x2*>(a.col_codes + (ca + 1) * (padded / 2) + r0 / 2) = u32x2{pb[0], pb[1]};
                a.col_scales[ca * (padded / 16) + r0 / 16] = (uint8_t)ba.code;
                a.col_scales[(ca + 1) * (padded / 16) + r0 / 16] = (uint8_t)bb.code;
            }
        }
    }
    if (a.amax) amax_commit(tmax, a.amax);
}

template <int TR, bool ROW, bool COL, bool SR, bool W32, bool ONCE>
void launch_as(const QuantizeGroupedArgs& a, hipStream_t stream) {
    const int64_t tiles = rows_padded(a.rows, a.experts) / TR * ((a.cols + kTileCols - 1) / kTileCols);
    in_launches(tiles, kThreads, [&](int64_t first, dim3 grid) {
        hipLaunchKernelGGL((quantize_grouped_kernel<TR, ROW, COL, SR, W32, ONCE>), grid, dim3(kThreads), 0, stream, a, first);
    });
}

template <int TR, bool ROW, bool COL, bool SR>
void launch(const QuantizeGroupedArgs& a, hipStream_t stream) {
    if constexpr (SR) {
        if (rows_padded(a.rows, a.experts) * a.cols < (int64_t)1 << 35)
            return a.index ? launch_as<TR, ROW, COL, SR, true, false>(a, stream) : launch_as<TR, ROW, COL, SR, true, true>(a, stream);
    }
    a.index ? launch_as<TR, ROW, COL, SR, false, false>(a, stream) : launch_as<TR, ROW, COL, SR, false, true>(a, stream);
}

}  // namespace

void launch_quantize_grouped(const QuantizeGroupedArgs& a, hipStream_t stream) {
    if (a.row_codes && a.col_codes)
        a.stochastic ? launch<64, true, true, true>(a, stream) : launch<64, true, true, false>(a, stream);
    else if (a.col_codes)
        a.stochastic ? launch<64, false, true, true>(a, stream) : launch<64, false, true, false>(a, stream);
    else if (a.row_codes)
        a.stochastic ? launch<32, true, false, true>(a, stream) : launch<32, true, false, false>(a, stream);
    else
        launch<32, false, false, false>(a, stream);
}

}  // namespace ue5m3fp4
