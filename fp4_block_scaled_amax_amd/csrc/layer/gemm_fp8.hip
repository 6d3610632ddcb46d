// 8-bit "NT" GEMM with one scale per block of 128 along K:
//   C[i][j] = sum_kb sA(i, kb) sB(j, kb) sum_{k in block kb} A(i, k) B(j, k)
// with E4M3 / E5M2 codes and fp32 or E8M0 scales (include/ue5m3fp4_layer.h).
#include "layer.hpp"

namespace ue5m3fp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kGroupM = 4;
constexpr int kSchedMfma = 0x008, kSchedValu = 0x002, kSchedDs = 0x100;

// How a block's scales reach the accumulators.
enum ScaleMode {
    kTileB,    // one scale per wave for B: a factor per lane
    kVectorB,  // one scale per row of B: a factor per element
    kHardware  // E8M0 scales as operands of the matrix instruction
};

__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int& tm, int& tn) {
    const int n = tiles_m * tiles_n;
    int id = blockIdx.x;
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

// The same address in every lane, as scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (const uint8_t*)(((uint64_t)hi << 32) | lo);
}

// 16 bytes per lane from base + off straight to LDS: lane l's at lds + 16 l.
// In assembly because the compiler, which cannot tell the two halves of the
// double buffer apart, would wait for the load at the next LDS read; it has no
// register output, and wait_staged() below waits for it.
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void wait_staged() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
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

// The scaled instruction; its byte selectors are immediates.
template <bool BE5, bool AE5>
__device__ __forceinline__ f32x4 mfma_scaled(int jb, int ib, i32x8 b, i32x8 a, f32x4 acc, uint32_t xb, uint32_t xa) {
#define UE5M3FP4_CASE(J, I)         \
    if (jb == J && ib == I)         \
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc, BE5, AE5, J, (int)xb, I, (int)xa);
#define UE5M3FP4_CASES(J) UE5M3FP4_CASE(J, 0) UE5M3FP4_CASE(J, 1) UE5M3FP4_CASE(J, 2) UE5M3FP4_CASE(J, 3)
    UE5M3FP4_CASES(0) UE5M3FP4_CASES(1) UE5M3FP4_CASES(2) UE5M3FP4_CASES(3)
#undef UE5M3FP4_CASES
#undef UE5M3FP4_CASE
    return acc;
}

template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0, int MW, int MI, int NI>
__global__ __launch_bounds__(MW * 128, 2) void gemm_fp8_kernel(GemmFp8Args g) {
    static_assert(SC != kHardware || (E8M0 && !EXACT), "hardware scales are E8M0 bytes of the 8-bit instruction");
    constexpr int kThreads = MW * 128, WM = 16 * MI, WN = 16 * NI, BM = MW * WM, BN = 2 * WN;
    constexpr int kStage = (BM + BN) * 128;
    typedef float scales_a __attribute__((ext_vector_type(MI)));
    __shared__ __align__(1024) uint8_t smem[2 * kStage];
    __shared__ __align__(16) float scales[2 * (BM + BN)];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int c = lane & 15, q = lane >> 4;

    int tm, tn;
    tile_of((int)((g.M + BM - 1) / BM), (int)((g.N + BN - 1) / BN), tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int64_t Kp = (g.K + 127) / 128 * 128;
    const int nchunks = (int)(Kp / 128);

    // ---- staging: one 1 KB load to LDS covers 8 rows x 128 codes; lane (r, p)
    // = (lane / 8, lane % 8) brings 16-byte unit p ^ (row / 2 % 8) of its row,
    // so that 16 rows' reads of one unit touch every bank once.  Offsets from
    // the tile's first code fit 32 bits (K < 2^24).
    constexpr int LA = BM / (16 * MW), LB = BN / (16 * MW);
    uint32_t oa[LA], ob[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int row = (wave * LA + i) * 8 + (lane >> 3);
        oa[i] = (uint32_t)min((int64_t)row, g.M - 1 - m0) * (uint32_t)Kp + 16 * ((lane & 7) ^ ((row >> 1) & 7));
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int row = (wave * LB + i) * 8 + (lane >> 3);
        ob[i] = (uint32_t)min((int64_t)row, g.N - 1 - n0) * (uint32_t)Kp + 16 * ((lane & 7) ^ ((row >> 1) & 7));
    }
    const uint8_t* ta = g.a.codes + m0 * Kp;
    const uint8_t* tb = g.b.codes + n0 * Kp;
    auto stage = [&](int k) __attribute__((always_inline)) {
        const uint32_t base = lds_address(smem) + (k & 1) * kStage;
        const uint8_t* ka = uniform(ta + (int64_t)k * 128);
        const uint8_t* kb = uniform(tb + (int64_t)k * 128);
#pragma unroll
        for (int i = 0; i < LA; ++i) load_lds16(ka, oa[i], base + (wave * LA + i) * 1024);
#pragma unroll
        for (int i = 0; i < LB; ++i) load_lds16(kb, ob[i], base + BM * 128 + (wave * LB + i) * 1024);
    };

    // ---- scales: thread t < BM + BN brings the scale of row t of A, then B,
    // a block ahead, and leaves it in LDS where the lanes read theirs at once:
    // A's as [16-row column c][tile i] of each wave row, B's by row (fp32) or
    // like A's (hardware).
    constexpr int kScaleBytes = E8M0 ? 1 : 4;
    const uint8_t* sp = nullptr;
    int64_t sstep = 0;
    int sput = 0;
    if (tid < BM) {
        const int64_t m = min(m0 + tid, g.M - 1);
        sstep = (g.a.tile ? (g.M + 127) / 128 : g.M) * kScaleBytes;
        sp = (const uint8_t*)g.a.scales + (g.a.tile ? m >> 7 : m) * kScaleBytes;
        sput = (tid / WM) * WM + (tid & 15) * MI + (tid % WM) / 16;
    } else if (tid < BM + BN) {
        const int r = tid - BM;
        const int64_t n = min(n0 + r, g.N - 1);
        sstep = (g.b.tile ? (g.N + 127) / 128 : g.N) * kScaleBytes;
        sp = (const uint8_t*)g.b.scales + (g.b.tile ? n >> 7 : n) * kScaleBytes;
        sput = SC == kHardware ? (r / WN) * WN + (r & 15) * NI + (r % WN) / 16 : r;
        sput += BM;
    }
    uint32_t sreg = 0u;
    auto load_scale = [&]() __attribute__((always_inline)) {
        if (BM + BN >= kThreads || tid < BM + BN) {
            if constexpr (E8M0) sreg = *sp;
            else sreg = *(const uint32_t*)sp;
            sp += sstep;
        }
    };
    auto put_scale = [&](int k) __attribute__((always_inline)) {
        if (BM + BN >= kThreads || tid < BM + BN) {
            if constexpr (SC == kHardware) ((uint8_t*)scales)[(k & 1) * (BM + BN) + sput] = (uint8_t)sreg;
            else scales[(k & 1) * (BM + BN) + sput] = E8M0 ? e8m0_value(sreg) : __uint_as_float(sreg);
        }
    };

    // ---- fragment reads: units 2q and 2q + 1 of row c (tile t: row 16 t + c)
    const int o0 = c * 128 + (((2 * q) ^ (c >> 1)) << 4), o1 = o0 ^ 16;
    const int a_base = wm * WM * 128, b_base = BM * 128 + wn * WN * 128;

    f32x4 acc[NI][MI];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (nchunks > 0) {
        stage(0);
        load_scale();
    }
    for (int k = 0; k < nchunks; ++k) {
        put_scale(k);
        wait_staged();  // this wave's share of chunk k is in LDS
        __syncthreads();
        if (k + 1 < nchunks) {
            stage(k + 1);
            load_scale();
        }
        const uint8_t* base = smem + (k & 1) * kStage;
        const float* sc = scales + (k & 1) * (BM + BN);

        Frag<EXACT, AE5> a[MI];
        Frag<EXACT, BE5> b[2];
        f32x4 part[2][MI], sv[2];
        scales_a fa;
        uint32_t xa = 0u;
        u32x2 xb = {0u, 0u};
        if constexpr (SC == kHardware) {
            const uint8_t* bytes = (const uint8_t*)scales + (k & 1) * (BM + BN);
            if constexpr (MI == 4) xa = *reinterpret_cast<const uint32_t*>(bytes + wm * WM + c * MI);
            else xa = *reinterpret_cast<const uint16_t*>(bytes + wm * WM + c * MI);
            if constexpr (NI == 8) xb = *reinterpret_cast<const u32x2*>(bytes + BM + wn * WN + c * NI);
            else xb.x = *reinterpret_cast<const uint32_t*>(bytes + BM + wn * WN + c * NI);
        } else {
            fa = *reinterpret_cast<const scales_a*>(sc + wm * WM + c * MI);
            if constexpr (SC == kTileB) fa *= sc[BM + wn * WN];
        }
        auto raw_b = [&](int j, i32x4& x, i32x4& y) __attribute__((always_inline)) {
            x = *reinterpret_cast<const i32x4*>(base + b_base + j * 2048 + o0);
            y = *reinterpret_cast<const i32x4*>(base + b_base + j * 2048 + o1);
        };
        auto read_sv = [&](int j) __attribute__((always_inline)) {
            if constexpr (SC == kVectorB) sv[j & 1] = *reinterpret_cast<const f32x4*>(sc + BM + wn * WN + 4 * q + 16 * j);
        };
        auto add_part = [&](int j, int i, const f32x4& p) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[j][i][e] = __builtin_fmaf(p[e], SC == kVectorB ? sv[j & 1][e] * fa[i] : fa[i], acc[j][i][e]);
        };
        i32x4 x, y;
        raw_b(0, x, y);
        b[0].set(x, y);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            a[i].set(*reinterpret_cast<const i32x4*>(base + a_base + i * 2048 + o0),
                     *reinterpret_cast<const i32x4*>(base + a_base + i * 2048 + o1));
        if constexpr (EXACT) {
            // widened fragments leave room for one of B and two partial sums
            f32x4 p[2];
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                if (j + 1 < NI) raw_b(j + 1, x, y);
                read_sv(j);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < 4; ++s) z = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[0].v[s], a[i].v[s], z, 0, 0, 0);
                    p[i & 1] = z;
                    if (i > 0) add_part(j, i - 1, p[(i - 1) & 1]);
                    else if (j > 0) add_part(j - 1, MI - 1, p[1]);
                }
                if (j + 1 < NI) b[0].set(x, y);
            }
            add_part(NI - 1, MI - 1, p[1]);
        } else {
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                if (j + 1 < NI) {
                    raw_b(j + 1, x, y);
                    b[(j + 1) & 1].set(x, y);
                }
                read_sv(j);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    if constexpr (SC == kHardware) {
                        // byte i of xa, byte j of xb
                        acc[j][i] = mfma_scaled<BE5, AE5>(j & 3, i, b[j & 1].v, a[i].v, acc[j][i], j < 4 ? xb.x : xb.y, xa);
                    } else {
                        f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                        part[j & 1][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j & 1].v, a[i].v, z, BE5, AE5, 0, 0, 0, 0);
                        if (j > 0) add_part(j - 1, i, part[(j - 1) & 1][i]);
                    }
                }
            }
            if constexpr (SC != kHardware) {
#pragma unroll
                for (int i = 0; i < MI; ++i) add_part(NI - 1, i, part[(NI - 1) & 1][i]);
            }
        }
        if constexpr (SC != kHardware && !EXACT) {
            __builtin_amdgcn_sched_group_barrier(kSchedDs, 3 + 2 * MI + (SC == kVectorB), 0);
#pragma unroll
            for (int t = 0; t < NI * MI; ++t) {
                __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
                if (t % MI == 0) __builtin_amdgcn_sched_group_barrier(kSchedDs, 2 + (SC == kVectorB), 0);
                __builtin_amdgcn_sched_group_barrier(kSchedValu, SC == kVectorB ? 8 : 4, 0);
            }
        }
    }

    // ---- epilogue: lane (c, q) holds columns n .. n + 3 of row m
    const bool vec = g.N % 4 == 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + wm * WM + 16 * i + c;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t n = n0 + wn * WN + 16 * j + 4 * q;
            const f32x4 v = acc[j][i];
            if (vec) {
                if (n >= g.N) continue;
                if (g.c_bf16)
                    *reinterpret_cast<bf16x4*>((__bf16*)g.c + m * g.N + n) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
                else
                    *reinterpret_cast<f32x4*>((float*)g.c + m * g.N + n) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (n + e >= g.N) continue;
                    if (g.c_bf16) ((__bf16*)g.c)[m * g.N + n + e] = (__bf16)v[e];
                    else ((float*)g.c)[m * g.N + n + e] = v[e];
                }
            }
        }
    }
}

template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0, int MW, int MI, int NI>
void launch_tiled(const GemmFp8Args& g, hipStream_t stream) {
    constexpr int BM = MW * 16 * MI, BN = 32 * NI;
    const int64_t tiles = ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
    hipLaunchKernelGGL((gemm_fp8_kernel<EXACT, AE5, BE5, SC, E8M0, MW, MI, NI>), dim3((unsigned)tiles), dim3(MW * 128), 0,
                       stream, g);
}

template <bool EXACT, bool AE5, bool BE5, int SC, bool E8M0>
void launch_size(const GemmFp8Args& g, hipStream_t stream) {
    const int64_t large = ((g.M + 255) / 256) * ((g.N + 255) / 256);
    if (large >= 192 && !EXACT) launch_tiled<EXACT, AE5, BE5, SC, E8M0, 4, 4, 8>(g, stream);
    else launch_tiled<EXACT, AE5, BE5, SC, E8M0, 2, 4, 4>(g, stream);
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
