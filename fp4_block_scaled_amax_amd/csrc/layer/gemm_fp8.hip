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

constexpr int kThreads = 512;
constexpr int kGroupM = 4;

// How a block's scales reach the accumulators.
enum ScaleMode {
    kTileB,    // fp32 (or decoded) scales, one per wave for B: a factor per lane
    kVectorB,  // fp32 (or decoded) scales, one per row of B: a factor per element
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

__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
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

template <bool EXACT, bool AE5, bool BE5, int SC, int MI, int NI>
__global__ __launch_bounds__(kThreads, 1) void gemm_fp8_kernel(GemmFp8Args g) {
    constexpr int BM = 64 * MI, BN = 32 * NI, WM = 16 * MI, WN = 16 * NI;
    constexpr int kStage = (BM + BN) * 128;
    __shared__ __align__(1024) uint8_t smem[2 * kStage];
    __shared__ __align__(16) float sb_lds[SC == kVectorB ? 2 * BN : 4];

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
    // so that 16 rows' reads of one unit touch every bank once.
    constexpr int LA = BM / 64, LB = BN / 64;
    const uint8_t* pa[LA];
    const uint8_t* pb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int row = (wave * LA + i) * 8 + (lane >> 3);
        pa[i] = g.a.codes + min(m0 + row, g.M - 1) * Kp + 16 * ((lane & 7) ^ ((row >> 1) & 7));
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int row = (wave * LB + i) * 8 + (lane >> 3);
        pb[i] = g.b.codes + min(n0 + row, g.N - 1) * Kp + 16 * ((lane & 7) ^ ((row >> 1) & 7));
    }
    auto stage = [&](int buf) __attribute__((always_inline)) {
        uint8_t* base = smem + buf * kStage;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            load_lds16(pa[i], base + (wave * LA + i) * 1024);
            pa[i] += 128;
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            load_lds16(pb[i], base + BM * 128 + (wave * LB + i) * 1024);
            pb[i] += 128;
        }
    };

    // ---- scales.  A: one per lane and 16-row tile (row c).  B: one per wave
    // (kTileB), or a row of BN in LDS (kVectorB), or one per lane and tile
    // (kHardware).
    const int64_t as_step = g.a.tile ? (g.M + 127) / 128 : g.M, bs_step = g.b.tile ? (g.N + 127) / 128 : g.N;
    int64_t as_at[MI], bs_at[SC == kHardware ? NI : 1];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = min(m0 + wm * WM + 16 * i + c, g.M - 1);
        as_at[i] = g.a.tile ? m >> 7 : m;
    }
    if constexpr (SC == kHardware) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t n = min(n0 + wn * WN + 16 * j + c, g.N - 1);
            bs_at[j] = g.b.tile ? n >> 7 : n;
        }
    } else if constexpr (SC == kTileB) {
        bs_at[0] = min(n0 + wn * WN, g.N - 1) >> 7;
    } else {
        const int64_t n = min(n0 + min(tid, BN - 1), g.N - 1);
        bs_at[0] = g.b.tile ? n >> 7 : n;
    }
    auto scale_f32 = [&](const void* base, int64_t at) __attribute__((always_inline)) {
        return g.e8m0 ? e8m0_value(((const uint8_t*)base)[at]) : ((const float*)base)[at];
    };
    float sa[MI], sb = 0.0f;
    int ha[MI], hb[SC == kHardware ? NI : 1];
    auto load_scales = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if constexpr (SC == kHardware) ha[i] = ((const uint8_t*)g.a.scales)[kb * as_step + as_at[i]];
            else sa[i] = scale_f32(g.a.scales, kb * as_step + as_at[i]);
        }
        if constexpr (SC == kHardware) {
#pragma unroll
            for (int j = 0; j < NI; ++j) hb[j] = ((const uint8_t*)g.b.scales)[kb * bs_step + bs_at[j]];
        } else {
            sb = scale_f32(g.b.scales, kb * bs_step + bs_at[0]);
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
        load_scales(0);
    }
    for (int k = 0; k < nchunks; ++k) {
        if constexpr (SC == kVectorB) {
            if (tid < BN) sb_lds[(k & 1) * BN + tid] = sb;
        }
        __builtin_amdgcn_s_waitcnt(0);  // this wave's share of chunk k (and its scales) is in LDS
        __syncthreads();
        float fa[MI];
        int xa[MI], xb[SC == kHardware ? NI : 1];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if constexpr (SC == kHardware) xa[i] = ha[i];
            else fa[i] = SC == kTileB ? sa[i] * sb : sa[i];
        }
        if constexpr (SC == kHardware) {
#pragma unroll
            for (int j = 0; j < NI; ++j) xb[j] = hb[j];
        }
        if (k + 1 < nchunks) {
            stage((k + 1) & 1);
            load_scales(k + 1);
        }
        const uint8_t* base = smem + (k & 1) * kStage;
        const float* sbv = sb_lds + (SC == kVectorB ? (k & 1) * BN + wn * WN + 4 * q : 0);
        Frag<EXACT, AE5> a[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i)
            a[i].set(*reinterpret_cast<const i32x4*>(base + a_base + i * 2048 + o0),
                     *reinterpret_cast<const i32x4*>(base + a_base + i * 2048 + o1));
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            Frag<EXACT, BE5> b;
            b.set(*reinterpret_cast<const i32x4*>(base + b_base + j * 2048 + o0),
                  *reinterpret_cast<const i32x4*>(base + b_base + j * 2048 + o1));
            f32x4 sv;
            if constexpr (SC == kVectorB) sv = *reinterpret_cast<const f32x4*>(sbv + 16 * j);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if constexpr (EXACT) {
                    f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(b.v[s], a[i].v[s], part, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[j][i][e] = __builtin_fmaf(part[e], SC == kVectorB ? sv[e] * fa[i] : fa[i], acc[j][i][e]);
                } else if constexpr (SC == kHardware) {
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a[i].v, acc[j][i], BE5, AE5, 0, xb[j],
                                                                                 0, xa[i]);
                } else {
                    f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
                    part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a[i].v, part, BE5, AE5, 0, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[j][i][e] = __builtin_fmaf(part[e], SC == kVectorB ? sv[e] * fa[i] : fa[i], acc[j][i][e]);
                }
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

template <bool EXACT, bool AE5, bool BE5, int SC>
void launch_size(const GemmFp8Args& g, hipStream_t stream) {
    const int64_t large = ((g.M + 255) / 256) * ((g.N + 255) / 256);
    if (large >= 192) {
        hipLaunchKernelGGL((gemm_fp8_kernel<EXACT, AE5, BE5, SC, 4, 8>), dim3((unsigned)large), dim3(kThreads), 0, stream, g);
    } else {
        const int64_t tiles = ((g.M + 127) / 128) * ((g.N + 127) / 128);
        hipLaunchKernelGGL((gemm_fp8_kernel<EXACT, AE5, BE5, SC, 2, 4>), dim3((unsigned)tiles), dim3(kThreads), 0, stream, g);
    }
}

template <bool AE5, bool BE5>
void launch_formats(const GemmFp8Args& g, hipStream_t stream) {
    if (!g.c_bf16) g.b.tile ? launch_size<true, AE5, BE5, kTileB>(g, stream) : launch_size<true, AE5, BE5, kVectorB>(g, stream);
    else if (g.e8m0) launch_size<false, AE5, BE5, kHardware>(g, stream);
    else g.b.tile ? launch_size<false, AE5, BE5, kTileB>(g, stream) : launch_size<false, AE5, BE5, kVectorB>(g, stream);
}

}  // namespace

void launch_gemm_fp8(const GemmFp8Args& g, hipStream_t stream) {
    if (g.a.e5m2) g.b.e5m2 ? launch_formats<true, true>(g, stream) : launch_formats<true, false>(g, stream);
    else g.b.e5m2 ? launch_formats<false, true>(g, stream) : launch_formats<false, false>(g, stream);
}

}  // namespace ue5m3fp4
