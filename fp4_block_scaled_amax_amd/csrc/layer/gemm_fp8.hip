// 8-bit "NT" GEMM with one scale per block of 128 along K:
//   C[i][j] = sum_kb sA(i, kb) sB(j, kb) sum_{k in block kb} A(i, k) B(j, k)
// with E4M3 / E5M2 codes and fp32 or E8M0 scales (include/ue5m3fp4_layer.h).
//
// Two arithmetics, by the type of the result.
//  - bf16: v_mfma_f32_16x16x128_f8f6f4, one instruction per tile and block.  Of
//    each 8 consecutive products it keeps what lies within 2^-13 of the largest
//    (measured with single products added to a cancelling pair); across those
//    groups it sums in fp32.  That is 0.8e-5 to 1.5e-5 of the result's norm on
//    normally distributed operands and 5e-5 to 9e-5 on heavy-tailed ones with
//    outlier columns, from K = 128 to 8192 alike, against 2e-3 for the rounding
//    to bf16 that follows.
//  - fp32: the codes widened to fp16, which holds every E4M3 and E5M2 value, and
//    v_mfma_f32_16x16x32_f16: exact products, fp32 sums (1e-7), at half the rate.
//    All 8-bit matrix instructions share the 13 bits, so no other one would do.
// Either way a block's sum enters the fp32 accumulators by one FMA per element
// with the block's scales; E8M0 scales of bf16 results are operands of the matrix
// instruction instead, and nothing is left to the vector ALU.
//
// The operands are exchanged (B first), so that a lane's scale of A is one value
// per tile and the four results it holds are four neighbouring columns of C: lane
// (c, q) = (lane % 16, lane / 16) supplies 32 codes of row c of each operand and
// holds columns 4 q .. 4 q + 3 of row c.  Which 32 of a row's 128 codes it has
// does not matter as long as both operands agree: they share the block's scale.
//
// Codes go from memory straight to LDS, a block (128 of K) ahead of the one that
// is multiplied; each wave multiplies MI x NI tiles.  launch_size() picks the
// workgroup's tile.
//
// Measured (cold operands, TFLOP/s of 2 M N K, +-3 % from card to card; the card's
// library runs 2980 in 8 bits with one scale per tensor and 1580 in fp16):
//   8192 x 16384 x 4096, bf16, fp32 scales    524 us  2100  MFMA busy 0.49 at 1.8
//       to 1.95 GHz, the vector ALU 0.40, waves waiting 0.37 of their time (the
//       4 FMAs per MFMA and lane alone would cost 9 to 17 %)
//   8192 x 4096 x 16384, bf16, E8M0 scales    426 us  2580  MFMA busy 0.57 at 1.9
//       to 2.0 GHz, vector ALU 0.21
//   4096 x 4096 x 8192, fp32, 1-D scales      250 us  1100  bound by the vector
//       ALU (0.67 busy: per MFMA 2 conversions and 2 steps of scaling)
//   1 x 16384 x 4096, bf16                     11.8 us  5.7 TB/s of B
#include "layer.hpp"

namespace ue5m3fp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kGroupM = 4;  // tile rows that are walked together

// How a block's scales reach the accumulators.
enum ScaleMode {
    kTileB,    // one scale per wave for B: a factor per lane
    kVectorB,  // one scale per row of B: a factor per element
    kHardware  // E8M0 scales as operands of the matrix instruction
};

// Workgroups are dealt to the 8 XCDs in turn: each takes a contiguous range of an
// order that walks kGroupM tile rows column by column, so that an L2 holds what
// its workgroups share.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int n = tiles_m * tiles_n;
    const int per_xcd = n / 8;
    if (id < per_xcd * 8) id = (id % 8) * per_xcd + id / 8;  // the tail keeps its id
    const int width = kGroupM * tiles_n;
    const int first_m = (id / width) * kGroupM;
    const int rows = min(tiles_m - first_m, kGroupM);
    tm = first_m + (id % width) % rows;
    tn = (id % width) / rows;
}

__device__ __forceinline__ float e8m0_value(uint32_t c) {
    return c == 0xFFu ? __uint_as_float(0x7FC00000u) : c == 0u ? 0x1p-127f : __uint_as_float(c << 23);
}

// Where a row keeps its eight 16-byte units: unit u at u ^ swizzle(row).  Two
// rows fill the 64 banks; the swizzle is one-to-one over 8 row pairs, so 16 rows'
// reads of one unit touch every bank once, and its values on row pairs 0, 1, 6, 7
// and on 2 .. 5 are each closed under ^ 2, so that the same holds where half of
// the rows read the unit two further, as a 16-byte read of all lanes makes them.
__device__ __forceinline__ int swizzle(int row) {
    const int t = row >> 1;
    return (t & 4) | ((t & 1) << 1) | (((t >> 1) ^ (t >> 2)) & 1);
}

// The same address in every lane, as scalar registers.  The s_nop is the wait of 5
// states that a vector memory instruction needs before it reads a scalar register
// that a vector instruction wrote; the compiler inserts it for its own
// instructions, but does not look into the assembly below.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t v = (uint64_t)p;
    uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    asm volatile("s_nop 4" : "+s"(lo), "+s"(hi));
    return (const uint8_t*)(((uint64_t)hi << 32) | lo);
}

// 16 bytes per lane from base + off straight to LDS: lane l's at lds + 16 l.
// In assembly because the compiler, which cannot tell the two halves of the
// double buffer apart, would wait for the load at the next LDS read; it has no
// register output, and wait_loads() below waits for it.  m0, which it writes, is
// an output because a clobber of a reserved register tells the compiler nothing
// (as an input, written by the compiler, the loads come later: 1 x 16384 x 4096
// 11.98 instead of 11.84 us).
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3" : "=&{m0}"(m0) : "s"(lds), "v"(off), "s"(base) : "memory");
}
// The same for one dword (or, zero-extended, one byte): lane l's at lds + 4 l.
template <bool BYTE>
__device__ __forceinline__ void load_lds_scale(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    if constexpr (BYTE)
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %2, %3" : "=&{m0}"(m0) : "s"(lds), "v"(off), "s"(base) : "memory");
    else
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, %3" : "=&{m0}"(m0) : "s"(lds), "v"(off), "s"(base) : "memory");
}
// Waits until at most N of this wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// 8 codes as fp16 (exact).
template <bool E5M2>
__device__ __forceinline__ f16x8 widen(int lo, int hi) {
    f16x8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int v = i < 2 ? lo : hi;
        f16x2 p;
        if constexpr (E5M2)
            p = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(v, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(v, 1.0f, false);
        else
            p = i & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, false);
        o[2 * i] = p.x;
        o[2 * i + 1] = p.y;
    }
    return o;
}

// A fragment of 16 rows x 128 codes: lane (c, q) = (lane % 16, lane / 16)
// holds 32 codes of row c.  EXACT: widened to fp16.
template <bool EXACT, bool E5M2>
struct Frag;
template <bool E5M2>
struct Frag<false, E5M2> {
    i32x8 v;
    __device__ __forceinline__ void set(i32x4 x, i32x4 y) { v = i32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}; }
};
template <bool E5M2>
struct Frag<true, E5M2> {
    f16x8 v[4];
    __device__ __forceinline__ void set(i32x4 x, i32x4 y) {
        v[0] = widen<E5M2>(x[0], x[1]);
        v[1] = widen<E5M2>(x[2], x[3]);
        v[2] = widen<E5M2>(y[0], y[1]);
        v[3] = widen<E5M2>(y[2], y[3]);
    }
};

// Columns n .. n + 3 of row m of C, those that exist.  With N no multiple of 4 the
// rows start at any element; a 16-byte (8-byte) store may do so too.
__device__ __forceinline__ void store4(const GemmFp8Args& g, int64_t m, int64_t n, f32x4 v) {
    const bf16x4 h = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    const int64_t at = m * g.N + n;
    if (n + 4 <= g.N) {
        if (g.c_bf16) __builtin_memcpy((__bf16*)g.c + at, &h, sizeof h);
        else __builtin_memcpy((float*)g.c + at, &v, sizeof v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        if (n + e >= g.N) continue;
        if (g.c_bf16) ((__bf16*)g.c)[at + e] = h[e];
        else ((float*)g.c)[at + e] = v[e];
    }
}

template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0, int MW, int MI, int NI, int STAGES, int KG>
__global__ __launch_bounds__(MW * 128 * KG, 2) void gemm_fp8_kernel(GemmFp8Args g) {
    static_assert(SC != kHardware || (E8M0 && !EXACT), "hardware scales are E8M0 bytes of the 8-bit instruction");
    constexpr int WM = 16 * MI, WN = 16 * NI, BM = MW * WM, BN = 2 * WN;
    constexpr int kCodes = (BM + BN) * 128, kStage = kCodes + (BM + BN) * 4;
    __shared__ __align__(1024) uint8_t smem_all[KG * STAGES * kStage];

    const int tid = threadIdx.x, lane = tid & 63;
    const int group = KG > 1 ? __builtin_amdgcn_readfirstlane(tid / (MW * 128)) : 0;
    const int wave = __builtin_amdgcn_readfirstlane(KG > 1 ? (tid >> 6) % (MW * 2) : tid >> 6);
    uint8_t* smem = smem_all + group * (STAGES * kStage);
    const int wm = wave >> 1, wn = wave & 1;
    const int c = lane & 15, q = lane >> 4;

    int tm, tn;
    tile_of((int)(blockIdx.x + g.first), (int)((g.M + BM - 1) / BM), (int)((g.N + BN - 1) / BN), tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int64_t Kp = (g.K + 127) / 128 * 128;
    // group g of KG takes blocks g, g + KG, ...; every group makes the same turns
    const int blocks = (int)(Kp / 128), turns = (blocks + KG - 1) / KG;
    const int nchunks = (blocks - group + KG - 1) / KG;

    // ---- staging: one 1 KB load to LDS covers 8 rows x 128 codes; lane (r, p)
    // = (lane / 8, lane % 8) brings 16-byte unit p ^ swizzle(row) of its row.
    // Offsets from the tile's first code fit 32 bits (K < 2^24).
    constexpr int LA = BM / (16 * MW), LB = BN / (16 * MW), kLoads = LA + LB + 1;
    uint32_t oa[LA], ob[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int row = (wave * LA + i) * 8 + (lane >> 3);
        oa[i] = (uint32_t)min((int64_t)row, g.M - 1 - m0) * (uint32_t)Kp + 16 * ((lane & 7) ^ swizzle(row));
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int row = (wave * LB + i) * 8 + (lane >> 3);
        ob[i] = (uint32_t)min((int64_t)row, g.N - 1 - n0) * (uint32_t)Kp + 16 * ((lane & 7) ^ swizzle(row));
    }
    const uint8_t* ta = g.a.codes + m0 * Kp;
    const uint8_t* tb = g.b.codes + n0 * Kp;
    // The scales follow, a dword per row of A, then B, 64 rows per load (waves
    // beyond those repeat one, so that every wave counts the same loads).
    constexpr int kScaleBytes = E8M0 ? 1 : 4, kScaleLoads = (BM + BN) / 64;
    const int sgroup = wave % kScaleLoads;
    const bool of_a = sgroup * 64 < BM;
    const Fp8Operand& so = of_a ? g.a : g.b;
    const int64_t srows = of_a ? g.M : g.N, sfirst = of_a ? m0 : n0;
    const int64_t sstep = (so.tile ? (srows + 127) / 128 : srows) * kScaleBytes;
    const int64_t srow = min(sfirst + sgroup * 64 - (of_a ? 0 : BM) + lane, srows - 1);
    const uint32_t os = (uint32_t)(so.tile ? (srow >> 7) - (sfirst >> 7) : srow - sfirst) * kScaleBytes;
    const uint8_t* ts = (const uint8_t*)so.scales + (so.tile ? sfirst >> 7 : sfirst) * kScaleBytes;
    auto stage = [&](int k, int buf) __attribute__((always_inline)) {
        const uint32_t base = lds_address(smem) + buf * kStage;
        const int64_t kblock = (int64_t)k * KG + group;
        const uint8_t* ka = uniform(ta + kblock * 128);
        const uint8_t* kb = uniform(tb + kblock * 128);
#pragma unroll
        for (int i = 0; i < LA; ++i) load_lds16(ka, oa[i], base + (wave * LA + i) * 1024);
#pragma unroll
        for (int i = 0; i < LB; ++i) load_lds16(kb, ob[i], base + BM * 128 + (wave * LB + i) * 1024);
        load_lds_scale<E8M0>(uniform(ts + kblock * sstep), os, base + kCodes + sgroup * 256);
    };

    // ---- fragment reads: units 2q and 2q + 1 of row c (tile t: row 16 t + c)
    const int o0 = c * 128 + (((2 * q) ^ swizzle(c)) << 4), o1 = o0 ^ 16;
    const int a_base = wm * WM * 128, b_base = BM * 128 + wn * WN * 128;

    f32x4 acc[NI][MI];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // The chunk loop.  kLate: a chunk's last column of tiles is multiplied after
    // the barrier that hands its buffer to the loads of chunk k + STAGES, between
    // the reads of the next chunk's first fragments, so that neither the barrier
    // nor the first reads leave the matrix cores idle (1024 x 4096 x 4096, one
    // workgroup per CU: 32.9 -> 26 us).  Widened fragments leave no registers to
    // hold them across the barrier (4096 x 4096 x 8192: 262 us, that way 272).
    constexpr bool kLate = !EXACT;
    auto value = [&](uint32_t w) __attribute__((always_inline)) { return E8M0 ? e8m0_value(w & 0xFFu) : __uint_as_float(w); };
    auto raw = [&](const uint8_t* tile, i32x4& x, i32x4& y) __attribute__((always_inline)) {
        x = *reinterpret_cast<const i32x4*>(tile + o0);
        y = *reinterpret_cast<const i32x4*>(tile + o1);
    };
    Frag<EXACT, AE5> a[MI];
    Frag<EXACT, BE5> b[EXACT ? 1 : 2];
    constexpr int kB1 = EXACT ? 0 : 1;  // b[j & kB1] holds column j
    f32x4 part[EXACT ? 1 : 2][EXACT ? 2 : MI], sv[2];
    float fa[MI], fa_next[MI];
    int xa[SC == kHardware ? MI : 1], xb[SC == kHardware ? NI : 1];
    int xa_next[SC == kHardware ? MI : 1], xb_next = 0;
    i32x4 x, y;

    auto read_scales = [&](const uint32_t* sc) __attribute__((always_inline)) {
        if constexpr (SC == kHardware) {
#pragma unroll
            for (int i = 0; i < MI; ++i) xa_next[i] = (int)sc[wm * WM + 16 * i + c];
#pragma unroll
            for (int j = 0; j < NI - 1; ++j) xb[j] = (int)sc[BM + wn * WN + 16 * j + c];
            xb_next = (int)sc[BM + wn * WN + 16 * (NI - 1) + c];  // the last column still needs its own
        } else {
            const float sb = SC == kTileB ? value(sc[BM + wn * WN]) : 1.0f;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                fa_next[i] = value(sc[wm * WM + 16 * i + c]);
                if constexpr (SC == kTileB) fa_next[i] *= sb;
            }
        }
    };
    auto take_scales = [&]() __attribute__((always_inline)) {
        if constexpr (SC == kHardware) {
#pragma unroll
            for (int i = 0; i < MI; ++i) xa[i] = xa_next[i];
            xb[NI - 1] = xb_next;
        } else {
#pragma unroll
            for (int i = 0; i < MI; ++i) fa[i] = fa_next[i];
        }
    };
    // the sums of tile (j, i) of the block into its accumulator
    auto add_part = [&](int j, int i) __attribute__((always_inline)) {
        const f32x4& p = EXACT ? part[0][i & 1] : part[j & 1][i];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[j][i][e] = __builtin_fmaf(p[e], SC == kVectorB ? sv[j & 1][e] * fa[i] : fa[i], acc[j][i][e]);
    };
    // tile (j, i) of the block; an earlier one's sums meanwhile: the tile a column
    // before, or, where widened fragments leave no room for a column, the last one
    auto multiply = [&](int j, int i) __attribute__((always_inline)) {
        if constexpr (SC == kHardware) {
            acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j & kB1].v, a[i].v, acc[j][i], BE5, AE5, 0, xb[j], 0, xa[i]);
        } else {
            f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (EXACT) {
#pragma unroll
                for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[j & kB1].v[s], a[i].v[s], z, 0, 0, 0);
                part[0][i & 1] = z;
                if (i > 0) add_part(j, i - 1);
                else if (j > 0) add_part(j - 1, MI - 1);
            } else {
                z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j & kB1].v, a[i].v, z, BE5, AE5, 0, 0, 0, 0);
                part[j & 1][i] = z;
                if (j > 0) add_part(j - 1, i);
                // in this order: brought together with the instruction that made
                // them, the sums would be waited for (fprop 544 -> 524 us)
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // this wave's share of chunk k is in LDS; of STAGES = 3 the next one stays in flight
    auto wait_chunk = [&](int k) __attribute__((always_inline)) {
        static_assert(STAGES == 2 || STAGES == 3, "at most one later block is in flight");
        if (STAGES == 3 && k + 1 < nchunks) wait_loads<kLoads>();
        else wait_loads<0>();
    };

    auto read_first = [&](const uint8_t* base) __attribute__((always_inline)) {
        read_scales(reinterpret_cast<const uint32_t*>(base + kCodes));
        raw(base + b_base, x, y);
        b[0].set(x, y);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            raw(base + a_base + i * 2048, x, y);
            a[i].set(x, y);
        }
    };

#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k)
        if (k < nchunks) stage(k, k);
    if (kLate && turns > 0) {
        if (nchunks > 0) wait_chunk(0);
        __syncthreads();
        if (STAGES - 1 < nchunks) stage(STAGES - 1, STAGES - 1);
        read_first(smem);
    }
    int buf = 0;
    for (int k = 0; k < turns; ++k) {
        if (KG > 1 && k >= nchunks) {  // the last turn of a group without a block: only its barrier
            __syncthreads();
            break;
        }
        const uint8_t* base = smem + buf * kStage;
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(base + kCodes);
        if constexpr (!kLate) {
            wait_chunk(k);
            __syncthreads();
            // every wave has read chunk k - 1: its buffer takes chunk k + STAGES - 1
            if (k + STAGES - 1 < nchunks) stage(k + STAGES - 1, buf == 0 ? STAGES - 1 : buf - 1);
            read_first(base);
        }
        take_scales();
        // the other workgroup's wave on the SIMD reads and converts meanwhile (4096 x
        // 4096 x 8192: 265 -> 256 us; waves that share their barriers gain nothing)
        if constexpr (EXACT && KG == 1) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            if (j + 1 < NI) {
                raw(base + b_base + (j + 1) * 2048, x, y);
                if constexpr (!EXACT) b[(j + 1) & 1].set(x, y);
            }
            if constexpr (SC == kVectorB) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(sc + BM + wn * WN + 4 * q + 16 * j);
#pragma unroll
                for (int e = 0; e < 4; ++e) sv[j & 1][e] = value(w[e]);
            }
            if (kLate && j + 1 == NI) break;
#pragma unroll
            for (int i = 0; i < MI; ++i) multiply(j, i);
            if constexpr (SC == kHardware) __builtin_amdgcn_sched_barrier(0);  // dgrad 436 -> 426 us
            if constexpr (EXACT) {
                if (j + 1 < NI) b[0].set(x, y);
            }
        }
        buf = buf == STAGES - 1 ? 0 : buf + 1;
        if constexpr (kLate) {
            // the sums up to here stay on this side of the barrier (left to itself
            // the compiler sinks them past it, and holds all they are made of)
#pragma unroll
            for (int j = 0; j < (SC == kHardware ? NI - 1 : NI - 2); ++j)
#pragma unroll
                for (int i = 0; i < MI; ++i) asm volatile("" : "+v"(acc[j][i]));
            // every read of chunk k is done: its buffer takes chunk k + STAGES
            if (k + 1 < nchunks) wait_chunk(k + 1);
            __syncthreads();
            if (k + STAGES < nchunks) stage(k + STAGES, buf == 0 ? STAGES - 1 : buf - 1);
            const uint8_t* next = smem + buf * kStage;  // behind the last chunk: read, not used
            read_scales(reinterpret_cast<const uint32_t*>(next + kCodes));
            raw(next + b_base, x, y);
            b[NI & 1].set(x, y);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                multiply(NI - 1, i);
                __builtin_amdgcn_sched_barrier(0);  // a[i]'s registers are free only now
                raw(next + a_base + i * 2048, x, y);
                a[i].set(x, y);
            }
            if constexpr (SC != kHardware) {
#pragma unroll
                for (int i = 0; i < MI; ++i) add_part(NI - 1, i);
            }
        } else {
            add_part(NI - 1, MI - 1);
            if constexpr (KG == 1) __builtin_amdgcn_s_setprio(0);
        }
    }

    if constexpr (KG > 1) {
        // the groups' sums meet in LDS, in the groups' order
        static_assert(NI * MI * 16 * MW * 128 * (KG - 1) <= KG * STAGES * kStage, "the sums fit the buffers");
        __syncthreads();
        f32x4* sums = reinterpret_cast<f32x4*>(smem_all) + (wave * 64 + lane);
        constexpr int kStep = MW * 128;
        if (group > 0) {
#pragma unroll
            for (int t = 0; t < NI * MI; ++t) sums[((group - 1) * NI * MI + t) * kStep] = acc[t / MI][t % MI];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g2 = 0; g2 < KG - 1; ++g2)
#pragma unroll
            for (int t = 0; t < NI * MI; ++t) acc[t / MI][t % MI] += sums[(g2 * NI * MI + t) * kStep];
    }

    // ---- epilogue: lane (c, q) holds columns n .. n + 3 of row m
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + wm * WM + 16 * i + c;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) store4(g, m, n0 + wn * WN + 16 * j + 4 * q, acc[j][i]);
    }
}

// Few rows of A (MT tiles of 16): the time is that of reading B once.  A workgroup
// owns 16 rows of B and all of A; its waves take every W-th block of K straight
// from memory (no wave shares another's codes, so LDS would only add a trip),
// several blocks in flight, and their sums meet in LDS in a fixed order.
template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0, int W, int MT>
__global__ __launch_bounds__(W * 64) void gemm_fp8_skinny_kernel(GemmFp8Args g) {
    constexpr int kDepth = MT == 1 ? 4 : 2;
    __shared__ __align__(16) f32x4 sums[MT][W][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t Kp = (g.K + 127) / 128 * 128;
    const int nchunks = (int)(Kp / 128);
    const int64_t as_step = g.a.tile ? (g.M + 127) / 128 : g.M, bs_step = g.b.tile ? (g.N + 127) / 128 : g.N;

    const uint8_t* pb = g.b.codes + min(n0 + c, g.N - 1) * Kp + 32 * q;
    const uint8_t* pa[MT];
    int64_t as_at[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = min((int64_t)(16 * i + c), g.M - 1);
        pa[i] = g.a.codes + m * Kp + 32 * q;
        as_at[i] = g.a.tile ? m >> 7 : m;
    }
    // this lane's rows of B: as an operand row (hardware scales), or as the
    // four output columns 4 q .. 4 q + 3
    constexpr int kSb = SC == kVectorB ? 4 : 1;
    int64_t bs_at[kSb];
#pragma unroll
    for (int e = 0; e < kSb; ++e) {
        const int64_t n = min(n0 + (SC == kHardware ? c : SC == kTileB ? 0 : 4 * q + e), g.N - 1);
        bs_at[e] = g.b.tile ? n >> 7 : n;
    }
    auto scale_at = [&](const void* base, int64_t at) __attribute__((always_inline)) {
        if constexpr (E8M0) return e8m0_value(((const uint8_t*)base)[at]);
        else return ((const float*)base)[at];
    };

    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = wave; k0 < nchunks; k0 += W * kDepth) {
        i32x4 bx[kDepth], by[kDepth], ax[kDepth][MT], ay[kDepth][MT];
        float sa[kDepth][MT], sb[kDepth][kSb];
        int ha[kDepth][MT], hb[kDepth];
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const int64_t k = min(k0 + d * W, nchunks - 1);  // past the end: read again, not used
            bx[d] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pb + k * 128));
            by[d] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pb + k * 128 + 16));
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                ax[d][i] = *reinterpret_cast<const i32x4*>(pa[i] + k * 128);
                ay[d][i] = *reinterpret_cast<const i32x4*>(pa[i] + k * 128 + 16);
                if constexpr (SC == kHardware) ha[d][i] = ((const uint8_t*)g.a.scales)[k * as_step + as_at[i]];
                else sa[d][i] = scale_at(g.a.scales, k * as_step + as_at[i]);
            }
            if constexpr (SC == kHardware) {
                hb[d] = ((const uint8_t*)g.b.scales)[k * bs_step + bs_at[0]];
            } else {
#pragma unroll
                for (int e = 0; e < kSb; ++e) sb[d][e] = scale_at(g.b.scales, k * bs_step + bs_at[e]);
            }
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            const bool used = k0 + d * W < nchunks;  // selected, not branched on: the loads stay ahead
            Frag<EXACT, BE5> b;
            b.set(bx[d], by[d]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                Frag<EXACT, AE5> a;
                a.set(ax[d][i], ay[d][i]);
                f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (SC == kHardware) {
                    z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, acc[i], BE5, AE5, 0, hb[d], 0, ha[d][i]);
                } else if constexpr (EXACT) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[s], a.v[s], z, 0, 0, 0);
                } else {
                    z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, z, BE5, AE5, 0, 0, 0, 0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (SC != kHardware) z[e] = __builtin_fmaf(z[e], sa[d][i] * sb[d][kSb == 4 ? e : 0], acc[i][e]);
                    acc[i][e] = used ? z[e] : acc[i][e];
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sums[i][wave][lane] = acc[i];
    __syncthreads();
    if (wave >= MT) return;  // wave i sums and stores tile i
    f32x4 v = sums[wave][0][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[wave][w][lane];
    if (16 * wave + c < g.M) store4(g, 16 * wave + c, n0 + 4 * q, v);
}

template <int MW, int MI, int NI>
int64_t tiles_of(const GemmFp8Args& g) {
    constexpr int BM = MW * 16 * MI, BN = 32 * NI;
    return ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
}

template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0, int MW, int MI, int NI, int STAGES, int KG>
void launch_tiled(const GemmFp8Args& g, hipStream_t stream) {
    constexpr int kThreads = MW * 128 * KG;
    in_launches(tiles_of<MW, MI, NI>(g), kThreads, [&](int64_t first, dim3 grid) {
        GemmFp8Args part = g;
        part.first = first;
        hipLaunchKernelGGL((gemm_fp8_kernel<EXACT, AE5, BE5, SC, E8M0, MW, MI, NI, STAGES, KG>), grid, dim3(kThreads), 0, stream, part);
    });
}

template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0, int MT>
void launch_skinny(const GemmFp8Args& g, hipStream_t stream) {
    constexpr int W = 8;
    hipLaunchKernelGGL((gemm_fp8_skinny_kernel<EXACT, AE5, BE5, SC, E8M0, W, MT>), dim3((unsigned)((g.N + 15) / 16)),
                       dim3(W * 64), 0, stream, g);
}

// The tile size is the one whose rounds of workgroups take the least time, by
// the time of a round over 4096 elements of K (us, measured; 256 CUs):
//                                              bf16 results   fp32 results
//   64 x 64, 1 per CU, K in 2 or 4 groups           12             13
//   64 x 64, 2 per CU, K in 2 groups                17             23
//   128 x 128, 1 per CU, K in 2 groups              26             36
//   128 x 128, 2 per CU                             35             65
//   256 x 256, 1 per CU                             65              -
// 512 x 4096 x 4096: 16.5 us, in 128 x 128 tiles 25; 1024 x 4096 x 4096: 26, in
// 64 x 64 32; 4096 x 4096 x 4096: 65, in 128 x 128 78.  K in groups: 1024 x 1024
// x 8192 (fp32) 25 us in 4 groups, 29 in 2, 36 in 1; 2048 x 2048 x 8192 72 in 2,
// 79 in 1; a bf16 row by 16384 x 4096 is bound by memory and best at 2 groups of
// 3 stages: 12.1, against 14.1 in 4 groups of 2.  Few rows of A go to the few-row
// kernel where small tiles would leave CUs idle: at most 16 with up to 255 tiles
// (1 x 4096 x 16384: 17 us against 37), at most 32 with up to 64 (21 x 3920 x
// 11523: 19 us against 27; at 128 tiles, 32 x 8192 x 4096, it is 15 against 11).
template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0>
void launch_size(const GemmFp8Args& g, hipStream_t stream) {
    const int64_t small = tiles_of<2, 2, 2>(g), medium = tiles_of<2, 4, 4>(g), large = tiles_of<4, 4, 8>(g);
    if (g.M <= 16 && small < 256) return launch_skinny<EXACT, AE5, BE5, SC, E8M0, 1>(g, stream);
    if (g.M <= 32 && small <= 64) return launch_skinny<EXACT, AE5, BE5, SC, E8M0, 2>(g, stream);
    const int64_t t_small = small <= 256 ? (EXACT ? 13 : 12) : (small + 511) / 512 * (EXACT ? 23 : 17);
    const int64_t t_medium = medium <= 256 ? (EXACT ? 36 : 26) : (medium + 511) / 512 * (EXACT ? 65 : 35);
    if constexpr (!EXACT)
        if ((large + 255) / 256 * 65 <= min(t_small, t_medium))
            return launch_tiled<EXACT, AE5, BE5, SC, E8M0, 4, 4, 8, 2, 1>(g, stream);
    if (t_medium <= t_small) {
        if (medium <= 256) return launch_tiled<EXACT, AE5, BE5, SC, E8M0, 2, 4, 4, 2, 2>(g, stream);
        return launch_tiled<EXACT, AE5, BE5, SC, E8M0, 2, 4, 4, 2, 1>(g, stream);
    }
    if (small > 256) return launch_tiled<EXACT, AE5, BE5, SC, E8M0, 2, 2, 2, 2, 2>(g, stream);
    launch_tiled<EXACT, AE5, BE5, SC, E8M0, 2, 2, 2, EXACT ? 2 : 3, EXACT ? 4 : 2>(g, stream);
}

template <bool EXACT, bool AE5, bool BE5, bool E8M0>
void launch_scales(const GemmFp8Args& g, hipStream_t stream) {
    if constexpr (E8M0 && !EXACT) launch_size<false, AE5, BE5, kHardware, true>(g, stream);
    else if (g.b.tile) launch_size<EXACT, AE5, BE5, kTileB, E8M0>(g, stream);
    else launch_size<EXACT, AE5, BE5, kVectorB, E8M0>(g, stream);
}

template <bool AE5, bool BE5>
void launch_formats(const GemmFp8Args& g, hipStream_t stream) {
    if (g.c_bf16) g.e8m0 ? launch_scales<false, AE5, BE5, true>(g, stream) : launch_scales<false, AE5, BE5, false>(g, stream);
    else g.e8m0 ? launch_scales<true, AE5, BE5, true>(g, stream) : launch_scales<true, AE5, BE5, false>(g, stream);
}

}  // namespace

void launch_gemm_fp8(const GemmFp8Args& g, hipStream_t stream) {
    if (g.a.e5m2) g.b.e5m2 ? launch_formats<true, true>(g, stream) : launch_formats<true, false>(g, stream);
    else g.b.e5m2 ? launch_formats<false, true>(g, stream) : launch_formats<false, false>(g, stream);
}

}  // namespace ue5m3fp4
