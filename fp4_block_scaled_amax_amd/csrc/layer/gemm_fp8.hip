// 8-bit "NT" GEMM with one scale per block of 128 along K:
//   C[i][j] = sum_kb sA(i, kb) sB(j, kb) sum_{k in block kb} A(i, k) B(j, k)
// with E4M3 / E5M2 codes and fp32 or E8M0 scales (include/ue5m3fp4_layer.h).
//
// The codes are widened to fp16, which holds every E4M3 and E5M2 value, and
// multiplied by v_mfma_f32_32x32x16_f16: lane (r, h) = (lane % 32, lane / 32)
// supplies 8 values of row r of each operand; accumulator register e of lane
// (r, h) holds row 8 (e / 4) + 4 h + e % 4 of the first operand and row r of
// the second.  Which 8 of the 16 a lane holds does not matter as long as both
// operands agree: a block of 128 has one scale.
//
// (The 8-bit matrix instructions do not sum in fp32: of each 8 consecutive
// products they keep what lies within 2^-13 of the largest -- 2e-5 to 4e-5 of
// the result's norm on random operands, against 1e-7 here.)
//
// A block's MFMAs sum into fresh registers, which enter the accumulators by
// one fp32 FMA per element with the block's scale: exact products, fp32 sums.
#include "layer.hpp"

namespace ue5m3fp4 {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;

__device__ __forceinline__ float scale_at(const Fp8Operand& o, bool e8m0, int64_t rows, int64_t row, int64_t kb) {
    const int64_t at = o.tile ? kb * ((rows + 127) / 128) + row / 128 : kb * rows + row;
    if (!e8m0) return ((const float*)o.scales)[at];
    const uint32_t c = ((const uint8_t*)o.scales)[at];
    return c == 0xFFu ? __uint_as_float(0x7FC00000u) : c == 0u ? 0x1p-127f : __uint_as_float(c << 23);
}

// 8 codes as fp16 (exact).
template <bool E5M2>
__device__ __forceinline__ f16x8 widen(u32x2 w) {
    f16x8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int v = (int)w[i >> 1];
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

// One wave computes 32 x 32 outputs, operands straight from memory.
template <bool AE5, bool BE5>
__global__ __launch_bounds__(kThreads) void gemm_fp8_kernel(GemmFp8Args g) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 31, h = lane >> 5;
    const int64_t tiles_n = (g.N + 63) / 64;
    const int64_t m0 = (blockIdx.x / tiles_n) * 64 + 32 * (wave >> 1), n0 = (blockIdx.x % tiles_n) * 64 + 32 * (wave & 1);
    const int64_t Kp = (g.K + 127) / 128 * 128;
    const int64_t ra = min(m0 + r, g.M - 1), rb = min(n0 + r, g.N - 1);
    const uint8_t* pa = g.a.codes + ra * Kp + 8 * h;
    const uint8_t* pb = g.b.codes + rb * Kp + 8 * h;
    f32x16 acc = {};
    for (int64_t kb = 0; kb < Kp / 128; ++kb) {
        f32x16 part = {};
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const f16x8 av = widen<AE5>(*reinterpret_cast<const u32x2*>(pa + kb * 128 + 16 * s));
            const f16x8 bv = widen<BE5>(*reinterpret_cast<const u32x2*>(pb + kb * 128 + 16 * s));
            part = __builtin_amdgcn_mfma_f32_32x32x16_f16(bv, av, part, 0, 0, 0);
        }
        const float sa = scale_at(g.a, g.e8m0, g.M, ra, kb);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int64_t n = min(n0 + 8 * (e >> 2) + 4 * h + (e & 3), g.N - 1);
            acc[e] = __builtin_fmaf(part[e], sa * scale_at(g.b, g.e8m0, g.N, n, kb), acc[e]);
        }
    }
    const int64_t m = m0 + r;
    if (m >= g.M) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int64_t n = n0 + 8 * (e >> 2) + 4 * h + (e & 3);
        if (n >= g.N) continue;
        if (g.c_bf16) ((__bf16*)g.c)[m * g.N + n] = (__bf16)acc[e];
        else ((float*)g.c)[m * g.N + n] = acc[e];
    }
}

}  // namespace

void launch_gemm_fp8(const GemmFp8Args& g, hipStream_t stream) {
    const int64_t tiles = ((g.M + 63) / 64) * ((g.N + 63) / 64);
    const dim3 grid((unsigned)tiles), block(kThreads);
    if (g.a.e5m2) {
        if (g.b.e5m2) hipLaunchKernelGGL((gemm_fp8_kernel<true, true>), grid, block, 0, stream, g);
        else hipLaunchKernelGGL((gemm_fp8_kernel<true, false>), grid, block, 0, stream, g);
    } else {
        if (g.b.e5m2) hipLaunchKernelGGL((gemm_fp8_kernel<false, true>), grid, block, 0, stream, g);
        else hipLaunchKernelGGL((gemm_fp8_kernel<false, false>), grid, block, 0, stream, g);
    }
}

}  // namespace ue5m3fp4
