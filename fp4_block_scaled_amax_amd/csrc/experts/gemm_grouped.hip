// The three GEMMs of routed experts' FP4 linears (gfx950):
//   fprop, dgrad: C[i][j] = tsA tsB_g sum_k A(i, k) B_g(j, k) for the rows i of
//                 expert g (A: grouped rows, B: expert weights)
//   wgrad:        C_g[i][j] = tsA tsB sum_p A(i, p) B(j, p) over the columns p
//                 of expert g (A, B: grouped transposed operands)
// on UE5M3/E2M1 block-16 operands ("UE5M3 FP4 Block Scaling for Stable Language
// Model Pretraining", abstract; "Rethinking Shrinkage Bias in LLM FP4
// Pretraining ... UFP4 Recipe", abstract: the three training GEMMs).
//
// Arithmetic.  gfx950's scaled FP4 matrix instruction takes neither UE5M3 scales
// nor blocks of 16, so each element is dequantized exactly to fp16, q s / 16 (at
// most 6 significant bits, within [2^-22, 43008], below 2^-14 on fp16's
// subnormal grid), and v_mfma_f32_32x32x16_f16 sums exact products in fp32; the
// epilogue multiplies by 256 tsA tsB.  Two elements cost v_cvt_scalef32_pk_f16_fp4
// (which applies 2^(max(e, 1) - 22), the exponent field of its fp32 operand) and
// v_pk_mul_f16 (by m = 8 + f, or f where e = 0): a scale byte (e, f) is expanded
// to one dword that holds both factors, the fp32 exponent above, fp16 m below.
//
// Tiles.  A workgroup of 4 waves computes 256 columns of up to 256 rows of one
// expert, in steps of 128 along the contraction, double-buffered in LDS.  The
// more rows a wave has the fewer conversions it does per matrix instruction (4
// VALU instructions at 128 x 128 per wave, 6 at 128 x 64, 8 at 64 x 64, 12 at 32 x
// 64), so an expert's rows go in tiles of 256 while more than 128 are left, and
// the rest in one tile of 128, 64 or 32 rows, whose four waves stand side by side.
// Full tiles are dealt first, the rests after them: the short ones fill what the
// last round of long ones leaves.
#include "../formats.hpp"
#include "experts.hpp"

namespace ue5m3fp4 {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBM = 256, kBN = 256, kBK = 128;
constexpr int kThreads = 256;
constexpr int kCodeStride = kBK / 2 + 8;  // 64 bytes per row, padded to 72
constexpr int kCodesA = 0;
constexpr int kCodesB = kCodesA + kBM * kCodeStride;
constexpr int kScaleBlockStride = kBM * 4 + 32;  // a block's 256 rows, padded
constexpr int kScalesA = kCodesB + kBN * kCodeStride;
constexpr int kScalesB = kScalesA + 8 * kScaleBlockStride;
constexpr int kStage = kScalesB + 8 * kScaleBlockStride;
constexpr int kLut = 2 * kStage;
constexpr int kSmem = kLut + 256 * 4;
constexpr int kGroupM = 4;  // tile rows that are walked together

// sched_group_barrier masks
constexpr int kSchedMfma = 0x008, kSchedValu = 0x002, kSchedDs = 0x300, kSchedVmemRead = 0x020;

// UE5M3 byte -> expanded dword (0xFF: m = NaN, which poisons what it enters).
__device__ __forceinline__ uint32_t expand_scale(uint32_t c) {
    const uint32_t e = c >> 3, f = c & 7u;
    const _Float16 m = c == kUe5m3Nan ? (_Float16)__builtin_nanf("") : (_Float16)(float)(e > 0u ? 8u + f : f);
    uint16_t mb;
    __builtin_memcpy(&mb, &m, 2);
    return ((max(e, 1u) + 105u) << 23) | (uint32_t)mb;
}

// 8 codes and their expanded scale -> 8 fp16 values q s / 16.
__device__ __forceinline__ f16x8_t dequant8(uint32_t w, uint32_t S) {
    const float sc = __uint_as_float(S);
    const uint16_t mb = (uint16_t)S;
    _Float16 m;
    __builtin_memcpy(&m, &mb, 2);
    const f16x2_t mm = {m, m};
    const f16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 0) * mm;
    const f16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 1) * mm;
    const f16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 2) * mm;
    const f16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, sc, 3) * mm;
    return f16x8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
    const __bf16 b = (__bf16)f;
    uint16_t u;
    __builtin_memcpy(&u, &b, 2);
    return u;
}

// A 16-byte unit (32 codes) of a row's step at k0.  Where K is no multiple of 128
// its halves are clamped into the row; blocks past K get the scale 0 below, whose
// factor m = 0 makes every code 0.
template <bool ALIGNED>
__device__ __forceinline__ u32x4 load_unit(const uint8_t* row, int64_t K, int64_t k0, int part) {
    if (ALIGNED) return *reinterpret_cast<const u32x4*>(row + k0 / 2 + 16 * part);
    const int64_t ka = min(k0 + 32 * part, K - 16), kb = min(k0 + 32 * part + 16, K - 16);
    const u32x2 x = *reinterpret_cast<const u32x2*>(row + ka / 2);
    const u32x2 y = *reinterpret_cast<const u32x2*>(row + kb / 2);
    return u32x4{x.x, x.y, y.x, y.y};
}

// The 8 scale bytes of a row's step at block b0.
template <bool ALIGNED>
__device__ __forceinline__ u32x2 load_scales(const uint8_t* row, int64_t blocks, int64_t b0) {
    if (ALIGNED) return *reinterpret_cast<const u32x2*>(row + b0);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t v = row[min(b0 + j, blocks - 1)];
        w[j >> 2] |= (b0 + j < blocks ? v : 0u) << (8 * (j & 3));
    }
    return u32x2{w[0], w[1]};
}

// What a workgroup computes: rows [0, rows) of A from `a` on times columns [0,
// cols) of B from `b` on; strides in bytes.
struct Tile {
    const uint8_t *a, *as, *b, *bs;
    int64_t a_stride, as_stride, b_stride, bs_stride;
    int64_t K;       // contraction; strides and K are a multiple of 128 where ALIGNED
    int rows, cols;  // of this tile, at least 1
    int64_t c;       // element offset of its first result
    float sa256, sb;
};

// Largest magnitude (bf16 bits) of the workgroup folded into *amax.
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

// One tile, by WM x WN waves of RI x CJ 32 x 32 results.  Lane (r, h) = (lane % 32,
// lane / 32) owns elements [64 h + 16 b, + 16) of each row's step in block-step b
// (0..3): one block, one scale, two matrix instructions.  A and B agree on it, so
// the sums are those of the plain order.  While a step's matrix instructions issue,
// the next step's operands are dequantized, the next block-step is read from LDS,
// chunk c + 1 is stored to LDS and chunk c + 2 loaded; the chunk's one barrier
// stands before its last block-step, whose operands are in registers.
template <int RI, int CJ, int WM, int WN, bool ALIGNED>
__device__ __forceinline__ void compute_tile(const Tile& t, uint8_t* smem, void* cptr, bool c_bf16, int64_t N,
                                             float* amax) {
    constexpr int kRows = 32 * RI * WM;
    constexpr int kUnitsA = (kRows + 63) / 64;  // 16-byte units per thread and chunk
    static_assert(32 * CJ * WN == kBN && WM * WN == 4, "4 waves, 256 columns");
    const uint32_t* lut = reinterpret_cast<const uint32_t*>(smem + kLut);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const int r = lane & 31, h = lane >> 5;
    const int nchunks = (int)((t.K + kBK - 1) / kBK);
    const int64_t blocks = t.K / 16;

    // Staging: thread tid takes part spart of rows srow + 64 i of both operands,
    // and the scales of row tid; rows past the tile are clamped (their results
    // are not stored).  The 16 lanes that an 8-byte LDS store serves per cycle
    // hold rows o, o + 1, o + 8, o + 9, which start 0, 18, 16 and 2 banks apart.
    const int sq = (tid >> 2) & 15, spart = tid & 3;
    const int srow = 16 * (tid >> 6) + 2 * (sq >> 2) + (sq & 1) + 8 * ((sq >> 1) & 1);
    const uint8_t* a_rows[kUnitsA];
    const uint8_t* b_rows[4];
#pragma unroll
    for (int i = 0; i < kUnitsA; ++i) a_rows[i] = t.a + min(srow + 64 * i, t.rows - 1) * t.a_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i) b_rows[i] = t.b + min(srow + 64 * i, t.cols - 1) * t.b_stride;
    const uint8_t* a_srow = t.as + min(tid, t.rows - 1) * t.as_stride;
    const uint8_t* b_srow = t.bs + min(tid, t.cols - 1) * t.bs_stride;
    const bool stage_a = kRows >= 64 || srow < kRows, scale_a = kRows >= kThreads || tid < kRows;

    // plain vector values, no arrays: they stay in registers
    u32x4 ra0, ra1, ra2, ra3, rb0, rb1, rb2, rb3;
    u32x2 rsa, rsb;
    auto gload = [&](int chunk) __attribute__((always_inline)) {
        const int64_t k0 = (int64_t)chunk * kBK;
        ra0 = load_unit<ALIGNED>(a_rows[0], t.K, k0, spart);
        if constexpr (kUnitsA > 1) ra1 = load_unit<ALIGNED>(a_rows[1], t.K, k0, spart);
        if constexpr (kUnitsA > 2) ra2 = load_unit<ALIGNED>(a_rows[2], t.K, k0, spart);
        if constexpr (kUnitsA > 3) ra3 = load_unit<ALIGNED>(a_rows[3], t.K, k0, spart);
        rb0 = load_unit<ALIGNED>(b_rows[0], t.K, k0, spart);
        rb1 = load_unit<ALIGNED>(b_rows[1], t.K, k0, spart);
        rb2 = load_unit<ALIGNED>(b_rows[2], t.K, k0, spart);
        rb3 = load_unit<ALIGNED>(b_rows[3], t.K, k0, spart);
        rsa = load_scales<ALIGNED>(a_srow, blocks, k0 / 16);
        rsb = load_scales<ALIGNED>(b_srow, blocks, k0 / 16);
    };
    auto lstore_codes = [&](uint8_t* base) __attribute__((always_inline)) {
        auto st = [](uint8_t* p, u32x4 v) __attribute__((always_inline)) {  // rows are 8-byte aligned
            *reinterpret_cast<u32x2*>(p) = v.xy;
            *reinterpret_cast<u32x2*>(p + 8) = v.zw;
        };
        uint8_t* pa = base + kCodesA + srow * kCodeStride + 16 * spart;
        uint8_t* pb = base + kCodesB + srow * kCodeStride + 16 * spart;
        if (stage_a) st(pa, ra0);
        if constexpr (kUnitsA > 1) st(pa + 64 * kCodeStride, ra1);
        if constexpr (kUnitsA > 2) st(pa + 128 * kCodeStride, ra2);
        if constexpr (kUnitsA > 3) st(pa + 192 * kCodeStride, ra3);
        st(pb, rb0);
        st(pb + 64 * kCodeStride, rb1);
        st(pb + 128 * kCodeStride, rb2);
        st(pb + 192 * kCodeStride, rb3);
    };
    uint32_t ea[8], eb[8];
    auto lut_fetch = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t wa = j < 4 ? rsa.x : rsa.y, wb = j < 4 ? rsb.x : rsb.y;
            ea[j] = lut[(wa >> (8 * (j & 3))) & 0xFFu];
            eb[j] = lut[(wb >> (8 * (j & 3))) & 0xFFu];
        }
    };
    auto lstore_scales = [&](uint8_t* base) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (scale_a) *reinterpret_cast<uint32_t*>(base + kScalesA + j * kScaleBlockStride + tid * 4) = ea[j];
            *reinterpret_cast<uint32_t*>(base + kScalesB + j * kScaleBlockStride + tid * 4) = eb[j];
        }
    };

    const int a_code_off = kCodesA + (wm * 32 * RI + r) * kCodeStride + 32 * h;
    const int b_code_off = kCodesB + (wn * 32 * CJ + r) * kCodeStride + 32 * h;
    const int a_sc_off = kScalesA + 4 * h * kScaleBlockStride + (wm * 32 * RI + r) * 4;
    const int b_sc_off = kScalesB + 4 * h * kScaleBlockStride + (wn * 32 * CJ + r) * 4;
    struct BlockStep {  // a lane's operands of 16 elements per row
        u32x2 ca[RI], cb[CJ];
        uint32_t sa[RI], sb[CJ];
    };
    struct Frags {
        f16x8_t a[RI], b[CJ];
    };
    auto read_bs = [&](BlockStep& s, const uint8_t* base, int b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            s.ca[i] = *reinterpret_cast<const u32x2*>(base + a_code_off + i * 32 * kCodeStride + 8 * b);
            s.sa[i] = *reinterpret_cast<const uint32_t*>(base + a_sc_off + b * kScaleBlockStride + i * 128);
        }
#pragma unroll
        for (int j = 0; j < CJ; ++j) {
            s.cb[j] = *reinterpret_cast<const u32x2*>(base + b_code_off + j * 32 * kCodeStride + 8 * b);
            s.sb[j] = *reinterpret_cast<const uint32_t*>(base + b_sc_off + b * kScaleBlockStride + j * 128);
        }
    };
    auto dequant = [&](Frags& f, const BlockStep& s, int half) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RI; ++i) f.a[i] = dequant8(half ? s.ca[i].y : s.ca[i].x, s.sa[i]);
#pragma unroll
        for (int j = 0; j < CJ; ++j) f.b[j] = dequant8(half ? s.cb[j].y : s.cb[j].x, s.sb[j]);
    };

    f32x16_t acc[RI][CJ];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    if (nchunks > 0) {
        gload(0);
        lut_fetch();
        lstore_codes(smem);
        lstore_scales(smem);
        gload(min(1, nchunks - 1));
        __syncthreads();

        BlockStep bsr[2];
        Frags fr[2];
        read_bs(bsr[0], smem, 0);
        dequant(fr[0], bsr[0], 0);

        for (int c = 0; c < nchunks; ++c) {
            uint8_t* cur = smem + (c & 1) * kStage;
            uint8_t* nxt = smem + ((c + 1) & 1) * kStage;
#pragma unroll
            for (int J = 0; J < 8; ++J) {
                const Frags& f = fr[J & 1];
#pragma unroll
                for (int i = 0; i < RI; ++i)
#pragma unroll
                    for (int j = 0; j < CJ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
                if (J == 0 || J == 2 || J == 4) read_bs(bsr[((J >> 1) + 1) & 1], cur, (J >> 1) + 1);
                if (J == 6) read_bs(bsr[0], nxt, 0);
                if (J == 1) {
                    lstore_codes(nxt);
                    lut_fetch();
                    gload(min(c + 2, nchunks - 1));
                }
                if (J == 2) lstore_scales(nxt);
                dequant(fr[(J + 1) & 1], bsr[((J + 1) >> 1) & 1], (J + 1) & 1);
                // each matrix instruction followed by its share of the rest
                constexpr int kMfmas = RI * CJ, kValu = 8 * (RI + CJ) / kMfmas + 1, kPer = 16 / kMfmas;
#pragma unroll
                for (int q = 0; q < kMfmas; ++q) {
                    __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(kSchedValu, kValu, 0);
                    if (q * kPer < 10) __builtin_amdgcn_sched_group_barrier(kSchedDs, 2 * kPer, 0);
                    if (q * kPer < 8) __builtin_amdgcn_sched_group_barrier(kSchedVmemRead, 2 * kPer, 0);
                }
                if (J == 5) __syncthreads();
            }
        }
    }

    // Epilogue: accumulator e of lane (r, h) is row 8 (e / 4) + 4 h + e % 4, column
    // r of its 32 x 32 tile.
    const int row0 = wm * 32 * RI + 4 * h, col0 = wn * 32 * CJ + r;
    const bool whole = t.rows == kRows && t.cols == kBN;
    float* C = (float*)cptr + t.c;
    uint16_t* Cb = (uint16_t*)cptr + t.c;
    uint32_t tmax = 0u;
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int row = row0 + i * 32 + 8 * (e >> 2) + (e & 3);
            const int64_t off = row * N + col0;
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
                if (whole || (row < t.rows && col0 + 32 * j < t.cols)) {
                    const float v = (acc[i][j][e] * t.sa256) * t.sb;
                    if (c_bf16) {
                        const uint16_t b = to_bf16(v);
                        Cb[off + j * 32] = b;
                        tmax = max(tmax, (uint32_t)(b & 0x7FFFu));
                    } else {
                        C[off + j * 32] = v;
                    }
                }
            }
        }
    if (amax) amax_commit(tmax, amax);
}

template <bool ALIGNED>
__device__ __forceinline__ void compute(const Tile& t, uint8_t* smem, const GemmGroupedArgs& g) {
    if (t.rows > 128) compute_tile<4, 4, 2, 2, ALIGNED>(t, smem, g.c, g.c_bf16, g.N, g.amax);
    else if (t.rows > 64) compute_tile<4, 2, 1, 4, ALIGNED>(t, smem, g.c, g.c_bf16, g.N, g.amax);
    else if (t.rows > 32) compute_tile<2, 2, 1, 4, ALIGNED>(t, smem, g.c, g.c_bf16, g.N, g.amax);
    else compute_tile<1, 2, 1, 4, ALIGNED>(t, smem, g.c, g.c_bf16, g.N, g.amax);
}

// Consecutive workgroups go to the 8 XCDs in turn: each takes a contiguous range
// of the n tiles, so that an L2 holds what its workgroups share.
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t n) {
    const int64_t per_xcd = n / 8;
    return id < per_xcd * 8 ? (id % 8) * per_xcd + id / 8 : id;  // the tail keeps its number
}

// Tile l of a tiles_m x tiles_n rectangle, kGroupM tile rows at a time.
__device__ __forceinline__ void tile_of(int64_t l, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
    const int64_t width = kGroupM * tiles_n, first_m = l / width * kGroupM;
    const int64_t rows = min(tiles_m - first_m, (int64_t)kGroupM);
    tm = first_m + l % width % rows;
    tn = l % width / rows;
}

// Expert of tile number id of fprop and dgrad, its rows, and the tile's number
// among the expert's full tiles (or -1 and the column tile, for the rest of its
// rows).  Every wave finds it for itself, 64 experts at a time.
struct Found {
    int g, begin, end;
    int64_t full_tile, tn;
};
__device__ __forceinline__ int full_tiles(int len) { return (len + kBM / 2 - 1) / kBM; }

__device__ __forceinline__ bool find_tile(const GemmGroupedArgs& a, int64_t id, int64_t tiles_n, Found& f) {
    const int lane = threadIdx.x & 63;
    int64_t full = 0, rest = 0;  // row tiles of each kind
    for (int base = 0; base < a.experts; base += 64) {
        int n = 0;
        bool more = false;
        if (base + lane < a.experts) {
            const GroupRows r = group_rows(a.offsets, base + lane, (int)a.rows);
            n = full_tiles(r.end - r.begin);
            more = r.end - r.begin > (int64_t)n * kBM;
        }
        full += __shfl(wave_scan(n), 63);
        rest += __popcll(__ballot(more));
    }
    const bool in_full = id < full * tiles_n;
    int64_t j = in_full ? id : id - full * tiles_n;
    if (!in_full && j >= rest * tiles_n) return false;
    j = xcd_order(j, (in_full ? full : rest) * tiles_n);
    int64_t before = 0;  // row tiles of this kind before `base`
    for (int base = 0; base < a.experts; base += 64) {
        GroupRows r{0, 0};
        int n = 0;
        if (base + lane < a.experts) {
            r = group_rows(a.offsets, base + lane, (int)a.rows);
            n = full_tiles(r.end - r.begin);
            if (!in_full) n = r.end - r.begin > (int64_t)n * kBM;
        }
        const int upto = wave_scan(n);
        const uint64_t votes = __ballot((before + upto) * tiles_n > j);
        if (votes) {
            const int l = __builtin_ctzll(votes);  // the first expert that reaches beyond j
            f.g = base + l;
            f.begin = __shfl(r.begin, l);
            f.end = __shfl(r.end, l);
            const int64_t local = j - (before + __shfl(upto - n, l)) * tiles_n;
            f.full_tile = in_full ? local : -1;
            f.tn = in_full ? 0 : local;
            return true;
        }
        before += __shfl(upto, 63);
    }
    return false;
}

template <bool ALIGNED>
__global__ __launch_bounds__(kThreads, 1) void gemm_grouped_nt_kernel(GemmGroupedArgs g) {
    __shared__ __align__(16) uint8_t smem[kSmem];
    Found f;
    const int64_t tiles_n = (g.N + kBN - 1) / kBN;
    if (!find_tile(g, g.first + blockIdx.x, tiles_n, f)) return;
    reinterpret_cast<uint32_t*>(smem + kLut)[threadIdx.x] = expand_scale(threadIdx.x);
    const int expert = __builtin_amdgcn_readfirstlane(f.g);
    const int begin = __builtin_amdgcn_readfirstlane(f.begin), end = __builtin_amdgcn_readfirstlane(f.end);
    const int full = full_tiles(end - begin);
    int64_t tm = full, tn = f.tn;
    if (f.full_tile >= 0) tile_of(f.full_tile, full, tiles_n, tm, tn);
    tm = __builtin_amdgcn_readfirstlane((int)tm);
    tn = __builtin_amdgcn_readfirstlane((int)tn);
    const int64_t m0 = begin + tm * kBM, n0 = tn * kBN;
    Tile t;
    t.a_stride = t.b_stride = g.K / 2;
    t.as_stride = t.bs_stride = g.K / 16;
    t.K = g.K;
    t.a = g.a_codes + m0 * t.a_stride;
    t.as = g.a_scales + m0 * t.as_stride;
    t.b = g.b_codes + (expert * g.N + n0) * t.b_stride;
    t.bs = g.b_scales + (expert * g.N + n0) * t.bs_stride;
    t.rows = (int)min(end - m0, (int64_t)kBM);
    t.cols = (int)min(g.N - n0, (int64_t)kBN);
    t.c = m0 * g.N + n0;
    t.sa256 = *g.a_ts * 256.0f;
    t.sb = g.b_ts[expert * g.b_ts_step];
    __syncthreads();  // scale table visible
    compute<ALIGNED>(t, smem, g);
}

__global__ __launch_bounds__(kThreads, 1) void gemm_grouped_wgrad_kernel(GemmGroupedArgs g) {
    __shared__ __align__(16) uint8_t smem[kSmem];
    reinterpret_cast<uint32_t*>(smem + kLut)[threadIdx.x] = expand_scale(threadIdx.x);
    const int64_t tiles_m = (g.M + kBM - 1) / kBM, tiles_n = (g.N + kBN - 1) / kBN;
    const int64_t j = xcd_order(g.first + blockIdx.x, g.experts * tiles_m * tiles_n);
    const int expert = (int)(j / (tiles_m * tiles_n));
    int64_t tm, tn;
    tile_of(j % (tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
    const GroupRows own = group_rows(g.offsets, expert, (int)g.rows);
    const int64_t padded = 128 * ((g.rows + 127) / 128 + g.experts), p = padded_begin(own.begin, expert);
    const int64_t m0 = tm * kBM, n0 = tn * kBN;
    Tile t;
    t.a_stride = t.b_stride = padded / 2;
    t.as_stride = t.bs_stride = padded / 16;
    t.K = ((int64_t)own.end - own.begin + 127) / 128 * 128;
    t.a = g.a_codes + m0 * t.a_stride + p / 2;
    t.as = g.a_scales + m0 * t.as_stride + p / 16;
    t.b = g.b_codes + n0 * t.b_stride + p / 2;
    t.bs = g.b_scales + n0 * t.bs_stride + p / 16;
    t.rows = (int)min(g.M - m0, (int64_t)kBM);
    t.cols = (int)min(g.N - n0, (int64_t)kBN);
    t.c = (expert * g.M + m0) * g.N + n0;
    t.sa256 = *g.a_ts * 256.0f;
    t.sb = *g.b_ts;
    __syncthreads();  // scale table visible
    compute<true>(t, smem, g);
}

}  // namespace

void launch_gemm_grouped_nt(const GemmGroupedArgs& args, hipStream_t stream) {
    GemmGroupedArgs g = args;
    // an expert's rows make at most rows / 256 tiles and one more
    const int64_t row_tiles = g.rows / kBM + (g.experts < g.rows ? g.experts : g.rows);
    in_launches(row_tiles * ((g.N + kBN - 1) / kBN), kThreads, [&](int64_t first, dim3 grid) {
        g.first = first;
        if (g.K % kBK == 0) hipLaunchKernelGGL(gemm_grouped_nt_kernel<true>, grid, dim3(kThreads), 0, stream, g);
        else hipLaunchKernelGGL(gemm_grouped_nt_kernel<false>, grid, dim3(kThreads), 0, stream, g);
    });
}

void launch_gemm_grouped_wgrad(const GemmGroupedArgs& args, hipStream_t stream) {
    GemmGroupedArgs g = args;
    const int64_t tiles = g.experts * ((g.M + kBM - 1) / kBM) * ((g.N + kBN - 1) / kBN);
    in_launches(tiles, kThreads, [&](int64_t first, dim3 grid) {
        g.first = first;
        hipLaunchKernelGGL(gemm_grouped_wgrad_kernel, grid, dim3(kThreads), 0, stream, g);
    });
}

}  // namespace ue5m3fp4
