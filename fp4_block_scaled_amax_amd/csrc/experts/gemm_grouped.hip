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
// Tiles.  A workgroup of 4 waves computes 128 columns of up to 256 (or 128) rows of
// one expert, in steps of 128 along the contraction, double-buffered in LDS; two
// workgroups share a CU, so that one converts while the other multiplies, and one
// loads its first step or stores its results while the other is in its loop.  The
// more rows a wave has the fewer conversions it does per matrix instruction (6 VALU
// instructions at 128 x 64 per wave, 8 at 64 x 64, 12 at 32 x 64), so an expert's
// rows go in tiles of full height while more than half of one is left, and the rest
// in one lower tile.  Full tiles are dealt first, the rests after them: the short
// ones fill what the last round of long ones leaves.
// Where that makes too few tiles for 256 CUs, 64 x 64 results whose contraction the
// waves share out.
#include "../formats.hpp"
#include "experts.hpp"

namespace ue5m3fp4 {

namespace {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBK = 128;
constexpr int kThreads = 256;
constexpr int kGroupM = 4;  // tile rows that are walked together

// A sum takes up to kChain steps (32768 elements, 2048 matrix instructions), each of
// which rounds it.  Where the terms are alike the roundings go one way: rows of one
// or two values each were off by up to 8e-6 of sum |a b| at 8192 elements, 4e-5 at 32768, 1e-4 at
// 65536 and 3e-3 at 2^21, random terms of one sign by 1e-6, 3e-6, 3e-6 and 3e-5.  Longer
// ones (LONG) are joined from sums of kFold steps, and what a join rounds off begins
// the next one, so that length adds nothing: 4e-6 at any.  That needs a second register
// for each sum, so such tiles have 128 rows: one expert's wgrad over 131072 rows, 4096 x
// 4096, 4.50 ms, 3.76 without; experts with shorter contractions beside it lose nothing.
constexpr int kChain = 256, kFold = 32;

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

// What a workgroup computes: rows [0, rows) of A from `a` on times columns [0,
// cols) of B from `b` on; strides in bytes.
struct Tile {
    const uint8_t *a, *as, *b, *bs;
    int64_t a_stride, as_stride, b_stride, bs_stride;
    int64_t K;       // contraction
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

// LDS accesses of a wave's lanes to each other's data: the hardware keeps a wave's in
// order, the compiler has to as well.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void put(float& to, float v, uint32_t&) { to = v; }
__device__ __forceinline__ void put(uint16_t& to, float v, uint32_t& tmax) {
    to = to_bf16(v);
    tmax = max(tmax, (uint32_t)(to & 0x7FFFu));
}

// A wave's results to C.  Stored from the accumulators an instruction writes 64-byte
// pieces of rows (bf16; 128 in fp32), and that bounds wide and short products; so
// each 32 rows pass through this wave's part of the staging buffers, which no one
// needs any more, and leave in 16 bytes per lane, whole rows of the wave's tile at a
// time: 16384 x 32768 results of bf16 stored alone take 255 us so, and 561 us without.
// They pass the caches, which then keep the operands (wgrad of 64 experts of 256 rows,
// 2048 x 4096, 594 -> 451 us).  Where rows of C do not begin at multiples of 16 bytes
// they are stored directly, in pieces that the caches join (past them 7 experts of 219
// rows, 2064 x 1305, would take 38 us instead of 26).  Returns the largest magnitude of
// what bf16 stores hold; rows and columns past the tile repeat its last ones, so they
// need no exception.
template <typename L, int RI, int CJ, typename OUT>
__device__ __forceinline__ uint32_t store_tile(const f32x16_t (&acc)[RI][CJ], const Tile& t, uint8_t* smem, OUT* C,
                                               int64_t N, int wm, int wn) {
    constexpr int kPer = 16 / sizeof(OUT), kLanes = 32 * CJ / kPer;  // results per lane, lanes per row
    constexpr int kStride = 32 * CJ * sizeof(OUT) + (sizeof(OUT) == 4 ? 32 : 16);  // rows 4 apart on other banks
    static_assert(32 * kStride <= L::kWave, "32 rows fit a wave's part");
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    uint8_t* mine = smem + (threadIdx.x >> 6) * L::kWave;
    const int row0 = wm * 32 * RI, col0 = wn * 32 * CJ;
    uint32_t tmax = 0u;
    C += t.c;
    if (N % kPer == 0) {
#pragma unroll
        for (int i = 0; i < RI; ++i) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
#pragma unroll
                for (int j = 0; j < CJ; ++j)
                    put(*reinterpret_cast<OUT*>(mine + (8 * (e >> 2) + 4 * h + (e & 3)) * kStride + (32 * j + r) * sizeof(OUT)),
                        (acc[i][j][e] * t.sa256) * t.sb, tmax);
            wave_sync();
#pragma unroll
            for (int m = 0; m < 32 * kLanes / 64; ++m) {
                const int row = m * (64 / kLanes) + lane / kLanes, col = lane % kLanes * kPer;
                const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * kStride + col * sizeof(OUT));
                if (row0 + 32 * i + row < t.rows && col0 + col < t.cols)
                    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(C + (row0 + 32 * i + row) * N + col0 + col));
            }
            wave_sync();
        }
        return tmax;
    }
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int row = row0 + i * 32 + 8 * (e >> 2) + 4 * h + (e & 3);
#pragma unroll
            for (int j = 0; j < CJ; ++j)
                if (row < t.rows && col0 + r + 32 * j < t.cols)
                    put(C[row * N + col0 + r + 32 * j], (acc[i][j][e] * t.sa256) * t.sb, tmax);
        }
    return tmax;
}

// 16 (4) bytes per lane from base + off straight to LDS, lane l's at lds + 16 l (4
// l).  In assembly, because the compiler would wait for them at every later LDS read;
// it knows neither the load nor when it ends: step_ready() does.  The s_nop is the
// wait that the load needs behind a vector instruction's write of its scalar base and
// behind that of m0, an output here because a clobber of it says nothing.
__device__ __forceinline__ void load_to_lds16(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %2, %3"
                 : "=&{m0}"(m0)
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void load_to_lds4(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dword %2, %3"
                 : "=&{m0}"(m0)
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base)
                 : "memory");
}
// This wave's loads have landed and its LDS reads are done; behind the barrier that
// holds for all waves: the step can be read, and the one before it overwritten.
__device__ __forceinline__ void step_ready() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// LDS of a workgroup with tiles of up to BM x 128: two steps of codes (64 bytes a
// row) and scale bytes (8 a row), and the table of expanded scales.
constexpr int kBN = 128;
template <int BM>
struct Lds {
    static_assert(BM >= 128, "4 waves bring the scales of 128 rows together");
    static constexpr int kCodesA = 0, kCodesB = BM * 64, kScalesA = kCodesB + kBN * 64, kScalesB = kScalesA + BM * 8;
    static constexpr int kStage = kScalesB + kBN * 8, kLut = 2 * kStage, kBytes = kLut + 1024;
    static constexpr int kWave = 32 * (64 * 4 + 32);  // a wave's part of it in the epilogue
    static_assert(4 * kWave <= kBytes, "the epilogue has room");
};

// 4 scale bytes of a row, from byte b on, where K is no multiple of 128: rows of scales
// begin anywhere.  Blocks past K get the scale 0, whose factor m = 0 makes every code
// 0.
typedef uint32_t u32_at1 __attribute__((aligned(1)));
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, uint32_t blocks, uint32_t b) {
    if (b + 4 <= blocks) return *reinterpret_cast<const u32_at1*>(row + b);
    uint32_t w = 0u;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        const uint32_t v = row[min(b + j, blocks - 1)];
        w |= (b + j < blocks ? v : 0u) << (8 * j);
    }
    return w;
}

template <int RI, int CJ>
__device__ __forceinline__ void fold_all(f32x16_t (&acc)[RI][CJ], f32x16_t (&sum)[RI][CJ]) {
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float s = sum[i][j][e];
                acc[i][j][e] = fold(s, acc[i][j][e]);
                sum[i][j][e] = s;
            }
}
template <int RI, int CJ>
__device__ __forceinline__ void add_all(f32x16_t (&acc)[RI][CJ], const f32x16_t (&sum)[RI][CJ]) {
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = sum[i][j][e] + acc[i][j][e];
}

// One tile of 32 RI WM rows x 128 columns, by WM x WN waves of RI x CJ 32 x 32
// results.
//
// A step's codes stand in LDS row by row, 64 bytes each, 16-byte unit u of row i at u
// ^ (i / 4 % 4), so that 16 lanes read a unit of 16 rows without bank conflicts.
// They come straight from memory, a step ahead of the one that is multiplied.  Where K
// is no multiple of 128 (not WHOLE) the last step's come in 4 bytes a lane, each
// clamped into its row, and scales through registers, since their rows begin anywhere
// then: the last step's are masked.
//
// Lane (r, h) = (lane % 32, lane / 32) owns elements [64 h, 64 h + 64) of a row's
// step: 2 units, 4 blocks, 8 matrix instructions.  A and B agree on it, so the sums
// are those of the plain order.  A scale byte is expanded where it is used: 16 rows'
// bytes mostly name few table entries.
template <int BM, int RI, int CJ, int WM, int WN, bool WHOLE, bool LONG>
__device__ __forceinline__ void compute_tile(const Tile& t, uint8_t* smem, const GemmGroupedArgs& g) {
    using L = Lds<BM>;
    constexpr int kRowsA = 32 * RI * WM;
    static_assert(32 * CJ * WN == kBN && kRowsA <= BM && WM * WN == 4, "4 waves, 128 columns");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r = lane & 31, h = lane >> 5;
    const int steps = __builtin_amdgcn_readfirstlane((int)((t.K + kBK - 1) / kBK));
    const uint32_t* lut = reinterpret_cast<const uint32_t*>(smem + L::kLut);

    // ---- staging: turn i of a wave brings the codes of rows 16 (wave + 4 i) .. + 15
    // (4 lanes a row) and the scales of rows 32 (wave + 4 i) .. + 31 (2 lanes a row);
    // rows past the tile repeat its last one, their results are not stored.  Offsets
    // fit 32 bits: 256 rows of less than 2^23 bytes.
    constexpr int kCodeTurnsA = (kRowsA + 63) / 64, kCodeTurnsB = kBN / 64, kScaleTurnsA = (kRowsA + 127) / 128;
    uint32_t oa[kCodeTurnsA], ob[kCodeTurnsB], osa[kScaleTurnsA], osb;
    const int code_row = 16 * wave + (lane >> 2), scale_row = 32 * wave + (lane >> 1);
    const uint32_t unit = (lane & 3) ^ ((code_row >> 2) & 3);  // rows 64 apart have the same
#pragma unroll
    for (int i = 0; i < kCodeTurnsA; ++i) oa[i] = (uint32_t)min(code_row + 64 * i, t.rows - 1) * (uint32_t)t.a_stride;
#pragma unroll
    for (int i = 0; i < kCodeTurnsB; ++i) ob[i] = (uint32_t)min(code_row + 64 * i, t.cols - 1) * (uint32_t)t.b_stride;
#pragma unroll
    for (int i = 0; i < kScaleTurnsA; ++i) osa[i] = (uint32_t)min(scale_row + 128 * i, t.rows - 1) * (uint32_t)t.as_stride;
    osb = (uint32_t)min(scale_row, t.cols - 1) * (uint32_t)t.bs_stride;
    const uint8_t *a = t.a, *as = t.as, *b = t.b, *bs = t.bs;  // scalar: so are all of a tile's values
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
    const uint32_t K = (uint32_t)t.K;
    auto stage = [&](int step, int at) __attribute__((always_inline)) {
        const uint32_t to = lds + at * L::kStage;
        const int64_t c = (int64_t)step * (kBK / 2), s = (int64_t)step * (kBK / 16);
        if (WHOLE || (uint32_t)(step + 1) * kBK <= K) {
#pragma unroll
            for (int i = 0; i < kCodeTurnsA; ++i)
                load_to_lds16(a + c, oa[i] + 16 * unit, to + L::kCodesA + 1024 * (wave + 4 * i));
#pragma unroll
            for (int i = 0; i < kCodeTurnsB; ++i) load_to_lds16(b + c, ob[i] + 16 * unit, to + L::kCodesB + 1024 * (wave + 4 * i));
        } else {  // 16 lanes a row, 4 rows a load
            const int sub_row = lane >> 4, sub = lane & 15;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const int row = 16 * wave + 4 * j + sub_row;
                const uint32_t k = min((uint32_t)step * (kBK / 2) + 16 * ((sub >> 2) ^ j) + 4 * (sub & 3), K / 2 - 4);
#pragma unroll
                for (int i = 0; i < kCodeTurnsA; ++i)
                    load_to_lds4(a, (uint32_t)min(row + 64 * i, t.rows - 1) * (uint32_t)t.a_stride + k,
                                 to + L::kCodesA + 1024 * (wave + 4 * i) + 256 * j);
#pragma unroll
                for (int i = 0; i < kCodeTurnsB; ++i)
                    load_to_lds4(b, (uint32_t)min(row + 64 * i, t.cols - 1) * (uint32_t)t.b_stride + k,
                                 to + L::kCodesB + 1024 * (wave + 4 * i) + 256 * j);
            }
        }
        if constexpr (WHOLE) {
#pragma unroll
            for (int i = 0; i < kScaleTurnsA; ++i)
                load_to_lds4(as + s, osa[i] + 4 * (lane & 1), to + L::kScalesA + 256 * (wave + 4 * i));
            load_to_lds4(bs + s, osb + 4 * (lane & 1), to + L::kScalesB + 256 * wave);
        }
    };
    uint32_t rsa[kScaleTurnsA], rsb;
    auto fetch_scales = [&](int step) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kScaleTurnsA; ++i) rsa[i] = load_scales(as + osa[i], K / 16, 8 * step + 4 * (lane & 1));
        rsb = load_scales(bs + osb, K / 16, 8 * step + 4 * (lane & 1));
    };
    auto put_scales = [&](int at) __attribute__((always_inline)) {
        uint8_t* to = smem + at * L::kStage;
#pragma unroll
        for (int i = 0; i < kScaleTurnsA; ++i)
            *reinterpret_cast<uint32_t*>(to + L::kScalesA + 256 * (wave + 4 * i) + 4 * lane) = rsa[i];
        *reinterpret_cast<uint32_t*>(to + L::kScalesB + 256 * wave + 4 * lane) = rsb;
    };

    const int row_a = wm * 32 * RI + r, row_b = wn * 32 * CJ + r;
    const int swizzle_a = (row_a >> 2) & 3, swizzle_b = (row_b >> 2) & 3;  // rows 32 apart have the same
    f32x16_t acc[RI][CJ], sum[LONG ? RI : 1][LONG ? CJ : 1];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                acc[i][j][e] = 0.0f;
                if constexpr (LONG) sum[i][j][e] = 0.0f;
            }

    if (steps > 0) {
        stage(0, 0);
        if constexpr (!WHOLE) {
            fetch_scales(0);
            put_scales(0);
        }
    }
    for (int step = 0; step < steps; ++step) {
        const uint8_t* cur = smem + (step & 1) * L::kStage;
        step_ready();
        if (step + 1 < steps) {
            stage(step + 1, (step + 1) & 1);
            if constexpr (!WHOLE) fetch_scales(step + 1);
        }
        uint32_t sa[RI], sb[CJ];
#pragma unroll
        for (int i = 0; i < RI; ++i) sa[i] = *reinterpret_cast<const uint32_t*>(cur + L::kScalesA + (row_a + 32 * i) * 8 + 4 * h);
#pragma unroll
        for (int j = 0; j < CJ; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(cur + L::kScalesB + (row_b + 32 * j) * 8 + 4 * h);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            u32x4 ca[RI], cb[CJ];
#pragma unroll
            for (int i = 0; i < RI; ++i)
                ca[i] = *reinterpret_cast<const u32x4*>(cur + L::kCodesA + (row_a + 32 * i) * 64 + 16 * ((2 * h + p) ^ swizzle_a));
#pragma unroll
            for (int j = 0; j < CJ; ++j)
                cb[j] = *reinterpret_cast<const u32x4*>(cur + L::kCodesB + (row_b + 32 * j) * 64 + 16 * ((2 * h + p) ^ swizzle_b));
#pragma unroll
            for (int block = 0; block < 2; ++block) {
                uint32_t ea[RI], eb[CJ];
#pragma unroll
                for (int i = 0; i < RI; ++i) ea[i] = lut[(sa[i] >> (8 * (2 * p + block))) & 0xFFu];
#pragma unroll
                for (int j = 0; j < CJ; ++j) eb[j] = lut[(sb[j] >> (8 * (2 * p + block))) & 0xFFu];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    f16x8_t fa[RI], fb[CJ];
#pragma unroll
                    for (int i = 0; i < RI; ++i) fa[i] = dequant8(ca[i][2 * block + s], ea[i]);
#pragma unroll
                    for (int j = 0; j < CJ; ++j) fb[j] = dequant8(cb[j][2 * block + s], eb[j]);
#pragma unroll
                    for (int i = 0; i < RI; ++i)
#pragma unroll
                        for (int j = 0; j < CJ; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
                }
            }
        }
        if constexpr (!WHOLE)
            if (step + 1 < steps) put_scales((step + 1) & 1);
        if constexpr (LONG)
            if (step % kFold == kFold - 1) fold_all(acc, sum);
    }
    if constexpr (LONG) add_all(acc, sum);
    step_ready();  // all waves are past their last step: the stages are free

    // Epilogue: accumulator e of lane (r, h) is row 8 (e / 4) + 4 h + e % 4, column
    // r of its 32 x 32 tile.
    uint32_t tmax = 0u;
    if (g.c_bf16) tmax = store_tile<L, RI, CJ, uint16_t>(acc, t, smem, (uint16_t*)g.c, g.N, wm, wn);
    else store_tile<L, RI, CJ, float>(acc, t, smem, (float*)g.c, g.N, wm, wn);
    if (g.amax) amax_commit(tmax, g.amax);
}

// The lowest tile that holds the rows: 64 unequal experts of 256 rows on average, 2048 ->
// 4096, 310 us, without the one of 192 rows 324.
template <int BM, bool WHOLE, bool LONG>
__device__ __forceinline__ void compute(const Tile& t, uint8_t* smem, const GemmGroupedArgs& g) {
    if constexpr (BM == 256 && !LONG) {
        if (t.rows > 192) return compute_tile<BM, 4, 2, 2, 2, WHOLE, LONG>(t, smem, g);
        if (t.rows > 128) return compute_tile<BM, 3, 2, 2, 2, WHOLE, LONG>(t, smem, g);
    }
    if (t.rows > 64) compute_tile<BM, 2, 2, 2, 2, WHOLE, LONG>(t, smem, g);
    else if (t.rows > 32) compute_tile<BM, 1, 2, 2, 2, WHOLE, LONG>(t, smem, g);
    else compute_tile<BM, 1, 1, 1, 4, WHOLE, LONG>(t, smem, g);
}

// A tile with a long contraction, 128 of its rows at a time.
template <int BM>
__device__ __forceinline__ void compute_long(const Tile& t, uint8_t* smem, const GemmGroupedArgs& g) {
#pragma unroll 1
    for (int m = 0; m < t.rows; m += 128) {
        Tile part = t;
        part.a += m * t.a_stride;
        part.as += m * t.as_stride;
        part.c += m * g.N;
        part.rows = min(t.rows - m, 128);
        if (m > 0) step_ready();  // the results before have left their place in LDS
        compute<BM, true, true>(part, smem, g);
    }
}

// ---- few tiles: the waves of a workgroup share out the contraction

// 16 bytes of codes of a row from element k on (a multiple of 32), K being no multiple
// of 128: blocks past K are clamped into the row.
typedef u32x4 u32x4_at8 __attribute__((aligned(8)));
__device__ __forceinline__ u32x4 load_codes(const uint8_t* row, uint32_t K, uint32_t k) {
    if (k + 32 <= K) return *reinterpret_cast<const u32x4_at8*>(row + k / 2);
    const u32x2 x = *reinterpret_cast<const u32x2*>(row + min(k, K - 16) / 2);
    const u32x2 y = *reinterpret_cast<const u32x2*>(row + min(k + 16, K - 16) / 2);
    return u32x4{x.x, x.y, y.x, y.y};
}

// One tile of 32 RI rows x 32 CJ columns: wave w takes steps w, w + 4, ... from memory
// to registers, a step ahead; then the waves' sums are joined in LDS, in a fixed
// order.
constexpr int kSplit = 4, kSplitRows = 64, kSplitCols = 64;
struct SplitLds {
    static constexpr int kRow = kSplitCols + 4, kLut = 4 * kSplit * kSplitRows * kRow, kBytes = kLut + 1024;  // floats of a row
};
template <int RI, int CJ>
struct Step {
    u32x4 ca[RI][2], cb[CJ][2];
    uint32_t sa[RI], sb[CJ];
};
template <int RI, int CJ, bool WHOLE, bool LONG>
__device__ __forceinline__ void split_tile(const Tile& t, uint8_t* smem, const GemmGroupedArgs& g) {
    using L = SplitLds;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t K = (uint32_t)t.K;
    const uint32_t* lut = reinterpret_cast<const uint32_t*>(smem + L::kLut);
    const uint8_t *a = t.a, *as = t.as, *b = t.b, *bs = t.bs;
    // rows past the tile repeat its last one, their results are not stored; a row's
    // scales begin at an eighth of its codes' offset
    uint32_t oa[RI], ob[CJ];
#pragma unroll
    for (int i = 0; i < RI; ++i) oa[i] = (uint32_t)min(32 * i + r, t.rows - 1) * (uint32_t)t.a_stride;
#pragma unroll
    for (int j = 0; j < CJ; ++j) ob[j] = (uint32_t)min(32 * j + r, t.cols - 1) * (uint32_t)t.b_stride;
    auto load = [&](Step<RI, CJ>& s, uint32_t k) __attribute__((always_inline)) {
        const uint32_t c = k / 2 + 32 * h;
        if (WHOLE || k + kBK <= K) {
#pragma unroll
            for (int i = 0; i < RI; ++i) {
#pragma unroll
                for (int p = 0; p < 2; ++p) s.ca[i][p] = *reinterpret_cast<const u32x4_at8*>(a + (oa[i] + c + 16 * p));
                s.sa[i] = *reinterpret_cast<const u32_at1*>(as + ((oa[i] + c) >> 3));
            }
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
#pragma unroll
                for (int p = 0; p < 2; ++p) s.cb[j][p] = *reinterpret_cast<const u32x4_at8*>(b + (ob[j] + c + 16 * p));
                s.sb[j] = *reinterpret_cast<const u32_at1*>(bs + ((ob[j] + c) >> 3));
            }
        } else {
#pragma unroll
            for (int i = 0; i < RI; ++i) {
#pragma unroll
                for (int p = 0; p < 2; ++p) s.ca[i][p] = load_codes(a + oa[i], K, k + 64 * h + 32 * p);
                s.sa[i] = load_scales(as + (oa[i] >> 3), K / 16, k / 16 + 4 * h);
            }
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
#pragma unroll
                for (int p = 0; p < 2; ++p) s.cb[j][p] = load_codes(b + ob[j], K, k + 64 * h + 32 * p);
                s.sb[j] = load_scales(bs + (ob[j] >> 3), K / 16, k / 16 + 4 * h);
            }
        }
    };
    f32x16_t acc[RI][CJ], sum[LONG ? RI : 1][LONG ? CJ : 1];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                acc[i][j][e] = 0.0f;
                if constexpr (LONG) sum[i][j][e] = 0.0f;
            }

    Step<RI, CJ> next;
    if (wave * kBK < K) load(next, wave * kBK);
    __syncthreads();  // the table of scales is there
    for (uint32_t k = wave * kBK; k < K; k += kSplit * kBK) {
        const Step<RI, CJ> cur = next;
        if (k + kSplit * kBK < K) load(next, k + kSplit * kBK);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int block = 0; block < 2; ++block) {
                uint32_t ea[RI], eb[CJ];
#pragma unroll
                for (int i = 0; i < RI; ++i) ea[i] = lut[(cur.sa[i] >> (8 * (2 * p + block))) & 0xFFu];
#pragma unroll
                for (int j = 0; j < CJ; ++j) eb[j] = lut[(cur.sb[j] >> (8 * (2 * p + block))) & 0xFFu];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    f16x8_t fa[RI], fb[CJ];
#pragma unroll
                    for (int i = 0; i < RI; ++i) fa[i] = dequant8(cur.ca[i][p][2 * block + s], ea[i]);
#pragma unroll
                    for (int j = 0; j < CJ; ++j) fb[j] = dequant8(cur.cb[j][p][2 * block + s], eb[j]);
#pragma unroll
                    for (int i = 0; i < RI; ++i)
#pragma unroll
                        for (int j = 0; j < CJ; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
                }
            }
        }
        if constexpr (LONG)
            if (k / (kSplit * kBK) % kFold == kFold - 1) fold_all(acc, sum);
    }
    if constexpr (LONG) add_all(acc, sum);

    // ---- the waves' sums: accumulator e of lane (r, h) is row 8 (e / 4) + 4 h + e % 4,
    // column r of its 32 x 32 tile
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                sums[(wave * 32 * RI + 32 * i + 8 * (e >> 2) + 4 * h + (e & 3)) * L::kRow + 32 * j + r] = acc[i][j][e];
    __syncthreads();
    // 4 columns per thread; columns come in fours where rows of C are aligned
    constexpr int kLanes = 32 * CJ / 4;
    uint32_t tmax = 0u;
#pragma unroll
    for (int m = 0; m < 32 * RI * kLanes / kThreads; ++m) {
        const int row = (m * kThreads + (int)threadIdx.x) / kLanes, col = 4 * (threadIdx.x % kLanes);
        f32x4_t v = *reinterpret_cast<const f32x4_t*>(sums + row * L::kRow + col);
#pragma unroll
        for (int w = 1; w < kSplit; ++w) v += *reinterpret_cast<const f32x4_t*>(sums + (w * 32 * RI + row) * L::kRow + col);
        if (row >= t.rows) continue;
        const int64_t to = t.c + row * g.N + col;
        if (g.c_bf16) {
            uint16_t o[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) put(o[d], (v[d] * t.sa256) * t.sb, tmax);
            uint16_t* C = (uint16_t*)g.c + to;
            if (g.N % 4 == 0) {
                if (col < t.cols) *reinterpret_cast<uint64_t*>(C) = (uint64_t)o[3] << 48 | (uint64_t)o[2] << 32 | (uint32_t)o[1] << 16 | o[0];
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (col + d < t.cols) C[d] = o[d];
            }
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) v[d] = (v[d] * t.sa256) * t.sb;
            float* C = (float*)g.c + to;
            if (g.N % 4 == 0) {
                if (col < t.cols) *reinterpret_cast<f32x4_t*>(C) = v;
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    if (col + d < t.cols) C[d] = v[d];
            }
        }
    }
    if (g.amax) amax_commit(tmax, g.amax);
}

// Consecutive workgroups go to the 8 XCDs in turn: each takes a contiguous range
// of the n tiles, so that an L2 holds what its workgroups share.
template <typename T>
__device__ __forceinline__ T xcd_order(T id, T n) {
    const T per_xcd = n / 8;
    return id < per_xcd * 8 ? (id % 8) * per_xcd + id / 8 : id;  // the tail keeps its number
}

// Tile l of a tiles_m x tiles_n rectangle, kGroupM tile rows at a time.
__device__ __forceinline__ void tile_of(uint32_t l, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t width = kGroupM * tiles_n, band = l / width, in = l - band * width;
    const uint32_t rows = min(tiles_m - band * kGroupM, (uint32_t)kGroupM);
    tn = in / rows;
    tm = band * kGroupM + in - tn * rows;
}

// Expert of tile number id of fprop and dgrad, its rows, and the tile's number
// among the expert's full tiles (or -1 and the column tile, for the rest of its
// rows).  Every wave finds it for itself, 64 experts at a time.
struct Found {
    int g, begin, end;
    bool full;
    uint32_t tile;  // number of a full tile among the expert's, or column tile
};
template <int SIZE>
__device__ __forceinline__ int full_tiles(int len) { return (int)(((uint32_t)len + (SIZE / 2 - 1)) / SIZE); }

// Tile numbers fit 32 bits: experts * N * K < 2^40 and K >= 16 where there are any.
template <int SIZE>
__device__ __forceinline__ bool find_tile(const GemmGroupedArgs& a, uint32_t id, uint32_t tiles_n, Found& f) {
    const int lane = threadIdx.x & 63;
    uint32_t full = 0, rest = 0;  // row tiles of each kind
    GroupRows r{0, 0};
    int n = 0;
    bool more = false;
    auto look = [&](int base) __attribute__((always_inline)) {
        r = GroupRows{0, 0};
        if (base + lane < a.experts) r = group_rows(a.offsets, base + lane, (int)a.rows);
        n = full_tiles<SIZE>(r.end - r.begin);
        more = (uint32_t)(r.end - r.begin) > (uint32_t)n * SIZE;
    };
    uint32_t upto = 0;
    for (int base = 0; base < a.experts; base += 64) {
        look(base);
        upto = wave_scan(n);
        full += __shfl((int)upto, 63);
        rest += __popcll(__ballot(more));
    }
    f.full = id < full * tiles_n;
    uint32_t j = f.full ? id : id - full * tiles_n;
    if (!f.full && j >= rest * tiles_n) return false;
    j = xcd_order(j, (f.full ? full : rest) * tiles_n);
    const uint32_t at = j / tiles_n;  // row tile of this kind
    uint32_t before = 0;
    for (int base = 0; base < a.experts; base += 64) {
        if (a.experts > 64) look(base);  // else still there
        if (!f.full) n = more;
        if (!f.full || a.experts > 64) upto = wave_scan(n);
        const uint64_t votes = __ballot(before + upto > at);
        if (votes) {
            const int l = __builtin_ctzll(votes);  // the first expert that reaches beyond
            f.g = base + l;
            f.begin = __shfl(r.begin, l);
            f.end = __shfl(r.end, l);
            f.tile = j - (before + __shfl((int)upto - n, l)) * tiles_n;
            return true;
        }
        before += __shfl((int)upto, 63);
    }
    return false;
}

// The tile of a workgroup of fprop and dgrad in tiles of up to BM x BN.
template <int BM, int BN>
__device__ __forceinline__ bool nt_tile(const GemmGroupedArgs& g, Tile& t) {
    Found f;
    const uint32_t tiles_n = (uint32_t)((g.N + BN - 1) / BN);
    if (!find_tile<BM>(g, (uint32_t)g.first + blockIdx.x, tiles_n, f)) return false;
    const int expert = __builtin_amdgcn_readfirstlane(f.g);
    const int begin = __builtin_amdgcn_readfirstlane(f.begin), end = __builtin_amdgcn_readfirstlane(f.end);
    const int full = full_tiles<BM>(end - begin);
    uint32_t tm = full, tn = __builtin_amdgcn_readfirstlane(f.tile);
    if (__builtin_amdgcn_readfirstlane(f.full)) tile_of(tn, full, tiles_n, tm, tn);
    const int64_t m0 = begin + (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    t.a_stride = t.b_stride = g.K / 2;
    t.as_stride = t.bs_stride = g.K / 16;
    t.K = g.K;
    t.a = g.a_codes + m0 * t.a_stride;
    t.as = g.a_scales + m0 * t.as_stride;
    t.b = g.b_codes + (expert * g.N + n0) * t.b_stride;
    t.bs = g.b_scales + (expert * g.N + n0) * t.bs_stride;
    t.rows = (int)min(end - m0, (int64_t)BM);
    t.cols = (int)min(g.N - n0, (int64_t)BN);
    t.c = m0 * g.N + n0;
    t.sa256 = scale_of_sum(*g.a_ts * 256.0f, t.K);
    t.sb = scale_of_sum(g.b_ts[expert * g.b_ts_step], t.K);
    return true;
}

// The tile of a workgroup of wgrad.
template <int BM, int BN>
__device__ __forceinline__ void wgrad_tile(const GemmGroupedArgs& g, Tile& t) {
    const uint32_t tiles_m = (uint32_t)((g.M + BM - 1) / BM), tiles_n = (uint32_t)((g.N + BN - 1) / BN);
    const uint32_t tiles = tiles_m * tiles_n;
    const int64_t id = g.first + blockIdx.x;
    const int expert = __builtin_amdgcn_readfirstlane((int)(id / tiles));
    // all XCDs share in every expert, whose rows may be many or few: 16384 rows of 8
    // unequal experts, 4096 x 4096, 515 us, 766 us where XCDs have experts of their own
    const uint32_t j = xcd_order((uint32_t)(id - (int64_t)expert * tiles), tiles);
    uint32_t tm, tn;
    tile_of(j, tiles_m, tiles_n, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    GroupRows own = group_rows(g.offsets, expert, (int)g.rows);
    own.begin = __builtin_amdgcn_readfirstlane(own.begin);
    own.end = __builtin_amdgcn_readfirstlane(own.end);
    const int64_t padded = 128 * ((g.rows + 127) / 128 + g.experts), p = padded_begin(own.begin, expert);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    t.a_stride = t.b_stride = padded / 2;
    t.as_stride = t.bs_stride = padded / 16;
    t.K = ((int64_t)own.end - own.begin + 127) / 128 * 128;
    t.a = g.a_codes + m0 * t.a_stride + p / 2;
    t.as = g.a_scales + m0 * t.as_stride + p / 16;
    t.b = g.b_codes + n0 * t.b_stride + p / 2;
    t.bs = g.b_scales + n0 * t.bs_stride + p / 16;
    t.rows = (int)min(g.M - m0, (int64_t)BM);
    t.cols = (int)min(g.N - n0, (int64_t)BN);
    t.c = (expert * g.M + m0) * g.N + n0;
    t.sa256 = scale_of_sum(*g.a_ts * 256.0f, t.K);
    t.sb = scale_of_sum(*g.b_ts, t.K);
}

template <int BM, bool WHOLE, bool LONG>
__global__ __launch_bounds__(kThreads, 2) void gemm_grouped_nt_kernel(GemmGroupedArgs g) {
    using L = Lds<BM>;
    __shared__ __align__(16) uint8_t smem[L::kBytes];
    Tile t;
    if (!nt_tile<BM, kBN>(g, t)) return;
    reinterpret_cast<uint32_t*>(smem + L::kLut)[threadIdx.x] = expand_scale(threadIdx.x);
    compute<BM, WHOLE, LONG>(t, smem, g);
}

// LONG: an expert may have more than kChain steps of rows.
template <int BM, bool LONG>
__global__ __launch_bounds__(kThreads, 2) void gemm_grouped_wgrad_kernel(GemmGroupedArgs g) {
    using L = Lds<BM>;
    __shared__ __align__(16) uint8_t smem[L::kBytes];
    reinterpret_cast<uint32_t*>(smem + L::kLut)[threadIdx.x] = expand_scale(threadIdx.x);
    Tile t;
    wgrad_tile<BM, kBN>(g, t);
    if constexpr (LONG)
        if (t.K > kChain * kBK) return compute_long<BM>(t, smem, g);
    compute<BM, true, false>(t, smem, g);
}

template <bool WHOLE, bool LONG>
__device__ __forceinline__ void split(const Tile& t, uint8_t* smem, const GemmGroupedArgs& g) {
    reinterpret_cast<uint32_t*>(smem + SplitLds::kLut)[threadIdx.x] = expand_scale(threadIdx.x);
    if (t.rows > 32) split_tile<2, 2, WHOLE, LONG>(t, smem, g);
    else split_tile<1, 2, WHOLE, LONG>(t, smem, g);
}

template <bool WHOLE, bool LONG>
__global__ __launch_bounds__(kThreads, LONG && !WHOLE ? 1 : 2) void gemm_grouped_nt_split_kernel(GemmGroupedArgs g) {
    __shared__ __align__(16) uint8_t smem[SplitLds::kBytes];
    Tile t;
    if (nt_tile<kSplitRows, kSplitCols>(g, t)) split<WHOLE, LONG>(t, smem, g);
}

template <bool LONG>
__global__ __launch_bounds__(kThreads, 2) void gemm_grouped_wgrad_split_kernel(GemmGroupedArgs g) {
    __shared__ __align__(16) uint8_t smem[SplitLds::kBytes];
    Tile t;
    wgrad_tile<kSplitRows, kSplitCols>(g, t);
    split<true, LONG>(t, smem, g);
}

template <int BM, int BN, typename KERNEL>
void launch_nt(GemmGroupedArgs g, hipStream_t stream, KERNEL kernel) {
    // an expert's rows make at most rows / BM tiles and one more
    const int64_t row_tiles = g.rows / BM + (g.experts < g.rows ? g.experts : g.rows);
    in_launches(row_tiles * ((g.N + BN - 1) / BN), kThreads, [&](int64_t first, dim3 grid) {
        g.first = first;
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, g);
    });
}

template <int BM, int BN, typename KERNEL>
void launch_wgrad(GemmGroupedArgs g, hipStream_t stream, KERNEL kernel) {
    const int64_t tiles = g.experts * ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
    in_launches(tiles, kThreads, [&](int64_t first, dim3 grid) {
        g.first = first;
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, g);
    });
}

// Two workgroups on each of the 256 CUs.
constexpr int64_t kFew = 512;

// Tiles of 64 x 64 with split contractions while all of them run at once: 4 experts of
// 128 rows, 4096 -> 2048 (256 of them), 38 -> 19 us, 4096 -> 4096 (512) 41 -> 32 us;
// 16 experts of 64 rows, 4096 -> 4096 (1024), would lose, 50 -> 57 us.  Tiles of 256
// rows where those are enough for all CUs: 8 experts of 1024 rows, 4096 -> 4096
// (1024), 264 -> 232 us; 8 of 512 rows, 4096 -> 2048 (256), would lose, 73 -> 78 us.
template <bool WHOLE>
void dispatch_nt(const GemmGroupedArgs& g, hipStream_t stream) {
    // tiles that experts with the mean number of rows make
    const int64_t some = g.experts < g.rows ? g.experts : g.rows, each = (g.rows + some - 1) / some;
    auto tiles = [&](int rows, int cols) { return some * ((each + rows - 1) / rows) * ((g.N + cols - 1) / cols); };
    if (tiles(kSplitRows, kSplitCols) <= kFew) {
        if (g.K > kSplit * kChain * kBK) launch_nt<kSplitRows, kSplitCols>(g, stream, gemm_grouped_nt_split_kernel<WHOLE, true>);
        else launch_nt<kSplitRows, kSplitCols>(g, stream, gemm_grouped_nt_split_kernel<WHOLE, false>);
    } else if (g.K > kChain * kBK) launch_nt<128, kBN>(g, stream, gemm_grouped_nt_kernel<128, WHOLE, true>);
    else if (tiles(256, kBN) < kFew) launch_nt<128, kBN>(g, stream, gemm_grouped_nt_kernel<128, WHOLE, false>);
    else launch_nt<256, kBN>(g, stream, gemm_grouped_nt_kernel<256, WHOLE, false>);
}

}  // namespace

void launch_gemm_grouped_nt(const GemmGroupedArgs& g, hipStream_t stream) {
    g.K % kBK == 0 ? dispatch_nt<true>(g, stream) : dispatch_nt<false>(g, stream);
}

// The same rule: one expert of 2048 rows, 1024 x 1024, 22 -> 11 us split; 4 experts of
// 512 rows, 1024 x 1024 (1024 tiles), would lose, 12 -> 16 us.  Tiles of 256 rows only
// where they have work beside their first loads and their results: 16 experts of 256
// rows, 2048 x 4096 (4096 tiles of 2 steps), 149 -> 137 us; 8 of 256, 2048 x 2048 (1024
// of 2), would lose, 32 -> 37 us, and 16 of 64, 2048 x 4096 (4096 of 1), 104 -> 115 us.
void launch_gemm_grouped_wgrad(const GemmGroupedArgs& g, hipStream_t stream) {
    auto tiles = [&](int rows, int cols) { return g.experts * ((g.M + rows - 1) / rows) * ((g.N + cols - 1) / cols); };
    const int64_t steps = (g.rows / g.experts + kBK - 1) / kBK;  // of an expert with the mean number of rows
    const int64_t most = (g.rows + kBK - 1) / kBK;  // steps of an expert with all rows
    if (tiles(kSplitRows, kSplitCols) <= kFew) {
        if (most > kSplit * kChain) launch_wgrad<kSplitRows, kSplitCols>(g, stream, gemm_grouped_wgrad_split_kernel<true>);
        else launch_wgrad<kSplitRows, kSplitCols>(g, stream, gemm_grouped_wgrad_split_kernel<false>);
    } else if (steps < 2 || tiles(256, kBN) < kFew || tiles(256, kBN) * steps < 10 * kFew) {
        if (most > kChain) launch_wgrad<128, kBN>(g, stream, gemm_grouped_wgrad_kernel<128, true>);
        else launch_wgrad<128, kBN>(g, stream, gemm_grouped_wgrad_kernel<128, false>);
    } else {
        if (most > kChain) launch_wgrad<256, kBN>(g, stream, gemm_grouped_wgrad_kernel<256, true>);
        else launch_wgrad<256, kBN>(g, stream, gemm_grouped_wgrad_kernel<256, false>);
    }
}

}  // namespace ue5m3fp4
