// Few bf16 tokens times UE5M3-FP4 weights (gfx950):
//   out[i][j] = ts_g sum_k x[i][k] W_g(j, k)
// with one weight matrix, or with the expert's that owns row i.
//
// Every weight byte is read once per 16 TT tokens, so what counts is to keep
// loads of them in flight and to convert them fast enough.  A workgroup owns 16 RT
// rows of W (columns of the result) and up to 16 TT tokens of one expert; its 8
// waves take steps of 256 along K in turn and join their sums in LDS, in a fixed
// order.  Lane (r, q) = (lane % 16, lane / 16) reads 64 consecutive codes (32 bytes,
// a whole 128-byte line by four lanes) and their 4 scale bytes of row r of each
// 16 x 16 tile, and the same 64 elements of token r, so the K order of the two
// operands of v_mfma_f32_16x16x32_bf16 agrees.
//
// q s has at most 6 significant bits and lies within [2^-18, 688128], so it is
// exact in bf16, and so are the products in fp32.
#include "../formats.hpp"
#include "experts.hpp"

namespace ue5m3fp4 {

namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kStep = 256;  // elements of K per wave and step

// Value of a UE5M3 byte; 0xFF: NaN.  The byte is the top of an fp32 number whose
// exponent bias is 112 larger, subnormals included.
__device__ __forceinline__ float scale_value(uint32_t c) {
    const float v = __uint_as_float(c << 20) * 0x1p112f;
    return c == kUe5m3Nan ? __uint_as_float(0x7FC00000u) : v;
}

// 8 codes times their scale, as bf16 (exact).
__device__ __forceinline__ bf16x8_t dequant8(uint32_t w, float s) {
    bf16x8_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2_t v = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0)
                          : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1)
                          : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2)
                                   : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
        o[2 * i] = (__bf16)(v[0] * s);
        o[2 * i + 1] = (__bf16)(v[1] * s);
    }
    return o;
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
    const __bf16 b = (__bf16)f;
    uint16_t u;
    __builtin_memcpy(&u, &b, 2);
    return u;
}

// Row block `slot` of the launch: its expert and rows.  Every wave finds it for
// itself, 64 experts at a time.
__device__ __forceinline__ bool find_rows(const WeightOnlyArgs& a, int64_t slot, int per_block, int& g, int& begin,
                                          int& end) {
    if (!a.offsets) {
        g = 0;
        begin = (int)(slot * per_block);
        end = (int)a.rows;
        return begin < end;
    }
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int base = 0; base < a.experts; base += 64) {
        GroupRows r{0, 0};
        if (base + lane < a.experts) r = group_rows(a.offsets, base + lane, (int)a.rows);
        const int n = (r.end - r.begin + per_block - 1) / per_block;
        const int upto = wave_scan(n);
        const uint64_t votes = __ballot(before + upto > slot);
        if (votes) {
            const int l = __builtin_ctzll(votes);
            g = base + l;
            begin = __shfl(r.begin, l) + (int)(slot - before - __shfl(upto - n, l)) * per_block;
            end = __shfl(r.end, l);
            return true;
        }
        before += __shfl(upto, 63);
    }
    return false;
}

// The 64 codes (8 dwords) and 4 scale bytes of one lane of a W tile, and 64
// elements of a token.  Where K is no multiple of 256 each block of 16 is clamped
// into the row; blocks past K get the scale 0 and tokens the value 0 there.
struct Codes {
    u32x4 lo, hi;
    uint32_t s;
};
template <bool ALIGNED>
__device__ __forceinline__ Codes load_codes(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t k) {
    Codes c;
    if (ALIGNED) {
        c.lo = *reinterpret_cast<const u32x4*>(codes + k / 2);
        c.hi = *reinterpret_cast<const u32x4*>(codes + k / 2 + 16);
        c.s = *reinterpret_cast<const uint32_t*>(scales + k / 16);
        return c;
    }
    u32x2 w[4];
    c.s = 0u;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int64_t kb = min(k + 16 * b, K - 16);
        w[b] = *reinterpret_cast<const u32x2*>(codes + kb / 2);
        c.s |= (k + 16 * b < K ? (uint32_t)scales[kb / 16] : 0u) << (8 * b);
    }
    c.lo = u32x4{w[0].x, w[0].y, w[1].x, w[1].y};
    c.hi = u32x4{w[2].x, w[2].y, w[3].x, w[3].y};
    return c;
}
template <bool ALIGNED>
__device__ __forceinline__ bf16x8_t load_x(const uint16_t* x, int64_t K, int64_t k) {
    u32x4 v;
    if (ALIGNED) {
        v = *reinterpret_cast<const u32x4*>(x + k);
    } else {
        v = *reinterpret_cast<const u32x4*>(x + min(k, K - 8));
        if (k >= K) v = u32x4{0u, 0u, 0u, 0u};
    }
    bf16x8_t o;
    __builtin_memcpy(&o, &v, 16);
    return o;
}

template <int RT, int TT, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void weight_only_kernel(WeightOnlyArgs a, int64_t tiles_n) {
    __shared__ f32x4_t sums[kWaves][RT][TT][64];
    const int64_t id = a.first + blockIdx.x;
    const int64_t slot = id / tiles_n, n0 = id % tiles_n * (16 * RT);
    int g, begin, end;
    if (!find_rows(a, slot, 16 * TT, g, begin, end)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;

    const uint8_t* codes[RT];
    const uint8_t* scales[RT];
    const uint16_t* x[TT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t row = g * a.N + min(n0 + 16 * i + r, a.N - 1);
        codes[i] = a.w_codes + row * (a.K / 2);
        scales[i] = a.w_scales + row * (a.K / 16);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) x[t] = a.x + min((int64_t)begin + 16 * t + r, (int64_t)end - 1) * a.ldx;

    f32x4_t acc[RT][TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[i][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    const int64_t steps = (a.K + kStep - 1) / kStep;
    Codes next[RT];
    if (wave < steps) {
#pragma unroll
        for (int i = 0; i < RT; ++i) next[i] = load_codes<ALIGNED>(codes[i], scales[i], a.K, (int64_t)wave * kStep + 64 * q);
    }
    for (int64_t c = wave; c < steps; c += kWaves) {
        const int64_t k = c * kStep + 64 * q;
        Codes now[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) now[i] = next[i];
        if (c + kWaves < steps) {
#pragma unroll
            for (int i = 0; i < RT; ++i) next[i] = load_codes<ALIGNED>(codes[i], scales[i], a.K, k + kWaves * kStep);
        }
        bf16x8_t xv[TT][8];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int u = 0; u < 8; ++u) xv[t][u] = load_x<ALIGNED>(x[t], a.K, k + 8 * u);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t w = u < 4 ? now[i].lo[u & 3] : now[i].hi[u & 3];
                const bf16x8_t wv = dequant8(w, scale_value((now[i].s >> (8 * (u >> 1))) & 0xFFu));
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv[t][u], acc[i][t], 0, 0, 0);
            }
    }

    // ---- join the waves' sums: lane (r, q) holds rows 4 q .. 4 q + 3 of W for token r
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) sums[wave][i][t][lane] = acc[i][t];
    __syncthreads();
    const float ts = a.w_ts[g * a.w_ts_step];
    for (int e = threadIdx.x; e < RT * TT * 64; e += kThreads) {
        const int l = e & 63, t = e / 64 % TT, i = e / 64 / TT;
        f32x4_t v = sums[0][i][t][l];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += sums[w][i][t][l];
        const int64_t row = (int64_t)begin + 16 * t + (l & 15), col = n0 + 16 * i + 4 * (l >> 4);
        if (row >= end) continue;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (col + d < a.N) {
                if (a.out_bf16) ((uint16_t*)a.out)[row * a.ldo + col + d] = to_bf16(v[d] * ts);
                else ((float*)a.out)[row * a.ldo + col + d] = v[d] * ts;
            }
        }
    }
}

template <int RT, int TT>
void launch(WeightOnlyArgs a, hipStream_t stream) {
    const int64_t tiles_n = (a.N + 16 * RT - 1) / (16 * RT);
    int64_t slots = (a.rows + 16 * TT - 1) / (16 * TT);
    if (a.offsets) slots = a.rows / (16 * TT) + (a.experts < a.rows ? a.experts : a.rows);
    in_launches(slots * tiles_n, kThreads, [&](int64_t first, dim3 grid) {
        a.first = first;
        if (a.K % kStep == 0) hipLaunchKernelGGL((weight_only_kernel<RT, TT, true>), grid, dim3(kThreads), 0, stream, a, tiles_n);
        else hipLaunchKernelGGL((weight_only_kernel<RT, TT, false>), grid, dim3(kThreads), 0, stream, a, tiles_n);
    });
}

}  // namespace

void launch_gemm_weight_only(const WeightOnlyArgs& a, hipStream_t stream) {
    if (a.rows <= 16) launch<2, 1>(a, stream);
    else launch<2, 4>(a, stream);
}

}  // namespace ue5m3fp4
