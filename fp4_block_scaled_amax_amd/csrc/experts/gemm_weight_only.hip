// Few bf16 tokens times UE5M3-FP4 weights (gfx950):
//   out[i][j] = ts_g sum_k x[i][k] W_g(j, k)
// with one weight matrix, or with the expert's that owns row i.
//
// Every weight byte is read once per block of tokens, so what counts is to keep
// loads of them in flight and to convert them fast enough.  A workgroup owns 16 RT
// rows of W (columns of the result) and the tokens of one expert, up to a limit;
// its waves share out K and join their sums in LDS, in a fixed order.  One token goes
// through dot products, more through v_mfma_f32_16x16x32_bf16, for which lane (r, q)
// = (lane % 16, lane / 16) has the same consecutive elements of row r of W and of token
// r, so the K order of the two operands agrees.
//
// q s has at most 6 significant bits and lies within [2^-18, 688128], so it is
// exact in bf16, and so are the products in fp32.
#include "../formats.hpp"
#include "experts.hpp"

namespace ue5m3fp4 {

namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// rows of codes begin at multiples of 8 bytes, rows of scales anywhere
typedef u32x4 u32x4_at8 __attribute__((aligned(8)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));
typedef uint16_t u16_at1 __attribute__((aligned(1)));

// 32 consecutive codes of a row and their 2 scale bytes.  In a step that K cuts
// short (`whole` false) each block of 16 is clamped into the row, and blocks past K
// get the scale 0.
struct Codes {
    u32x4 w;
    uint32_t s;
};
__device__ __forceinline__ void load_codes(Codes& c, const uint8_t* codes, const uint8_t* scales, uint32_t row,
                                           uint32_t K, uint32_t k, bool whole) {
    if (__builtin_expect(whole, 1)) {
        const uint32_t at = row * (K / 2) + k / 2;
        c.w = *reinterpret_cast<const u32x4_at8*>(codes + at);
        c.s = *reinterpret_cast<const u16_at1*>(scales + (at >> 3));
        return;
    }
    c.s = 0u;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t at = row * (K / 16) + min(k + 16 * b, K - 16) / 16;
        const u32x2 v = *reinterpret_cast<const u32x2*>(codes + at * 8);
        c.w[2 * b] = v.x;
        c.w[2 * b + 1] = v.y;
        c.s |= (k + 16 * b < K ? (uint32_t)scales[at] : 0u) << (8 * b);
    }
}

// 8 elements of a token, zeros past K.
__device__ __forceinline__ bf16x8_t load_x(const uint16_t* x, uint32_t K, uint32_t k, bool whole) {
    u32x4 v = *reinterpret_cast<const u32x4*>(x + (whole ? k : min(k, K - 8)));
    if (!whole && k >= K) v = u32x4{0u, 0u, 0u, 0u};
    bf16x8_t o;
    __builtin_memcpy(&o, &v, 16);
    return o;
}

// Scale byte b of s times 2^-112: the byte is the top of an fp32 number whose
// exponent bias is 112 larger, subnormals included.  0xFF is NaN; whether a wave
// has one is asked once for all its bytes.
__device__ __forceinline__ float scale_value(uint32_t s, int b) {
    const uint32_t at20 = b == 0 ? s << 20 : b == 1 ? s << 12 : b == 2 ? s << 4 : s >> 4;
    return __uint_as_float(at20 & 0x0FF00000u);
}
__device__ __forceinline__ bool any_nan(uint32_t s) {  // a byte of s is 0xFF: a byte of ~s is 0
    return ((~s - 0x01010101u) & s & 0x80808080u) != 0u;
}

// 8 codes times their scale, as bf16 (exact): the conversion brings the 2^112.
__device__ __forceinline__ bf16x8_t dequant8(uint32_t w, float s) {
    bf16x8_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2_t v = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 0x1p112f, 0)
                          : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 0x1p112f, 1)
                          : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 0x1p112f, 2)
                                   : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 0x1p112f, 3);
        o[2 * i] = (__bf16)(v[0] * s);
        o[2 * i + 1] = (__bf16)(v[1] * s);
    }
    return o;
}

// The same without their scale, times 8 elements of a token over 128, added to `sum`:
// 16 products of the largest elements with the largest codes stay finite.
__device__ __forceinline__ float dot8(uint32_t w, bf16x8_t x, float sum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2_t v = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 0x1p-7f, 0)
                           : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 0x1p-7f, 1)
                           : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 0x1p-7f, 2)
                                    : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 0x1p-7f, 3);
        sum = __builtin_amdgcn_fdot2_f32_bf16(v, bf16x2_t{x[2 * i], x[2 * i + 1]}, sum, false);
    }
    return sum;
}

// The value of the lane D before this one, around the 16 lanes of a row.
template <int D>
__device__ __forceinline__ float rotated(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x120 + D, 0xF, 0xF, false));
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
    const __bf16 b = (__bf16)f;
    uint16_t u;
    __builtin_memcpy(&u, &b, 2);
    return u;
}

// K up to which a wave's sum takes its terms one after another: at most 512 matrix
// instructions (4 waves), whose roundings come to 3e-5 of sum |x w| where rows hold one or
// two values each (random terms of one sign: 1e-6).  Beyond (LONG: 2e-4 and 1e-5 at 2^23)
// sums of kFold are joined, and what a join rounds off begins the next one: 8e-6.  16
// tokens, 131072 -> 4096, 130 us, 100 without.
constexpr int64_t kChain = 65536;
constexpr uint32_t kFold = 32;  // steps of 128 (128 matrix instructions), or chunks of a token

// Where a launch's workgroups begin: row block `slot`, column tile `tile` of `tiles`.
struct Place {
    int64_t slot;
    uint32_t tile, tiles;
};

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
        const int n = (int)(((uint32_t)(r.end - r.begin) + (uint32_t)(per_block - 1)) / (uint32_t)per_block);
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

// One token per workgroup.  16 lanes share a row of W: each has 32 consecutive
// codes of a chunk of 512 (a row's 256 bytes are read together) and the same 32
// elements of the token, which it keeps in registers for all rows.  The waves
// share out the chunks.  Products in v_dot2_f32_bf16, which with the conversion to
// bf16 costs one instruction per weight, where the matrix instruction would need
// the scale in its operand, another one; the scale enters once per block.  4096 ->
// 16384 (37.7 MB) takes 8.7 us, an empty launch 2.4 us, and a kernel that only reads
// those bytes in the same pattern 6.7 us: bound by the loads' latency and bandwidth.
template <int ROWS, int WAVES, bool WHOLE, bool LONG>
__global__ __launch_bounds__(64 * WAVES, 4) void one_token_kernel(WeightOnlyArgs a, Place place) {
    constexpr int kLoads = ROWS / 4;  // 4 rows of W per load
    __shared__ float sums[WAVES][ROWS];
    const uint32_t u0 = place.tile + blockIdx.x, down = u0 / place.tiles;
    const int64_t slot = place.slot + down, n0 = (int64_t)(u0 - down * place.tiles) * ROWS;
    int g, begin, end;
    if (!find_rows(a, slot, 1, g, begin, end)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    begin = __builtin_amdgcn_readfirstlane(begin);
    const float ts = scale_of_sum(a.w_ts[g * a.w_ts_step], a.K);
    const int lane = threadIdx.x & 63, l = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t K = (uint32_t)a.K;
    const int rows = (int)min(a.N - n0, (int64_t)ROWS);
    const uint8_t* codes = a.w_codes + (g * a.N + n0) * (a.K / 2);
    const uint8_t* scales = a.w_scales + (g * a.N + n0) * (a.K / 16);
    const uint16_t* x = a.x + begin * a.ldx;

    float sum[kLoads], total[LONG ? kLoads : 1];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        sum[i] = 0.0f;
        if constexpr (LONG) total[i] = 0.0f;
    }
    bf16x8_t xnext[4];
    Codes next[kLoads];
    auto load = [&](uint32_t k0) __attribute__((always_inline)) {
        const uint32_t k = k0 + 32 * l;
        const bool whole = WHOLE || k0 + 512 <= K;
#pragma unroll
        for (int u = 0; u < 4; ++u) xnext[u] = load_x(x, K, k + 8 * u, whole);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_codes(next[i], codes, scales, (uint32_t)min(4 * i + q, rows - 1), K, k, whole);
    };
    if (wave * 512 < K) load(wave * 512);
    for (uint32_t k0 = wave * 512; k0 < K; k0 += WAVES * 512) {
        bf16x8_t xv[4];
        Codes c[kLoads];
#pragma unroll
        for (int u = 0; u < 4; ++u) xv[u] = xnext[u];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) c[i] = next[i];
        if (k0 + WAVES * 512 < K) load(k0 + WAVES * 512);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            float s0 = scale_value(c[i].s, 0), s1 = scale_value(c[i].s, 1);
            if (__builtin_expect(__any(any_nan(c[i].s)), 0)) {
                if ((c[i].s & 0xFFu) == kUe5m3Nan) s0 = __uint_as_float(0x7FC00000u);
                if ((c[i].s >> 8) == kUe5m3Nan) s1 = __uint_as_float(0x7FC00000u);
            }
            const float d0 = dot8(c[i].w[1], xv[1], dot8(c[i].w[0], xv[0], 0.0f));
            const float d1 = dot8(c[i].w[3], xv[3], dot8(c[i].w[2], xv[2], 0.0f));
            sum[i] = __builtin_fmaf(d0, s0 * 0x1p119f, sum[i]);
            sum[i] = __builtin_fmaf(d1, s1 * 0x1p119f, sum[i]);
            if constexpr (LONG)
                if (k0 / (WAVES * 512) % kFold == kFold - 1) sum[i] = fold(total[i], sum[i]);
        }
    }
    if constexpr (LONG) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) sum[i] = total[i] + sum[i];
    }

    // the 16 lanes of a row, then the waves, in a fixed order
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        sum[i] += rotated<8>(sum[i]);
        sum[i] += rotated<4>(sum[i]);
        sum[i] += rotated<2>(sum[i]);
        sum[i] += rotated<1>(sum[i]);
        if (l == 0) sums[wave][4 * i + q] = sum[i];
    }
    __syncthreads();
    if ((int)threadIdx.x < rows) {
        float v = sums[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += sums[w][threadIdx.x];
        const int64_t at = begin * a.ldo + n0 + threadIdx.x;
        if (a.out_bf16) ((uint16_t*)a.out)[at] = to_bf16(v * ts);
        else ((float*)a.out)[at] = v * ts;
    }
}

// 16 bytes per lane from base + off straight to LDS, lane l's at lds + 16 l.  In
// assembly, because the compiler would wait for them at every later LDS read; it
// knows neither the load nor when it ends: loads_done() does.  The s_nop is the wait
// that the load needs behind a vector instruction's write of its scalar base and
// behind that of m0, an output here because a clobber of it says nothing.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t off, uint32_t lds) {
    uint32_t m0;
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %2, %3"
                 : "=&{m0}"(m0)
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void lds_reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Up to TOKENS tokens (4, or a multiple of 16), 16 RT rows of W: v_mfma_f32_16x16x32_
// bf16 on codes converted with their scale.  In steps of 128 lane (r, q) = (lane %
// 16, lane / 16) has 32 consecutive codes of row r and the same 32 elements of token
// r.  A wave brings its own step's tokens to LDS, in whole lines, while it multiplies
// the step before; unit u (16 bytes) of token t stands at u ^ (t % 16) of the
// token's 256 bytes, since without it 16 tokens would meet in the same banks.  Two
// still do (a 16-byte read serves lanes 0-3, 12-15 and 20-27 together); places
// without any conflict changed no time.  64 tokens, 4096 -> 16384: 26 us, where loads straight
// to registers took 74 us; bound by the conversions (2 instructions a weight), by the
// tokens' reads, which every workgroup repeats, and by the weights: a row block's next
// codes go into the registers of the ones just multiplied, so the last block's are asked for
// right before the wait for the tokens, and arrive while nothing is multiplied.
template <int RT, int TOKENS, int WAVES, bool WHOLE, bool LONG>
__global__ __launch_bounds__(64 * WAVES, TOKENS > 32 ? 2 : 4) void tokens_kernel(WeightOnlyArgs a, Place place) {
    constexpr int kStep = 128, kUnits = 16;  // elements of K, and units of a token, per step
    constexpr int TT = (TOKENS + 15) / 16;
    constexpr int kTokenBytes = WAVES * TOKENS * kUnits * 16, kSumBytes = WAVES * RT * TT * 64 * 16;
    __shared__ __align__(16) uint8_t smem[kTokenBytes > kSumBytes ? kTokenBytes : kSumBytes];
    const uint32_t u0 = place.tile + blockIdx.x, down = u0 / place.tiles;
    const int64_t slot = place.slot + down, n0 = (int64_t)(u0 - down * place.tiles) * (16 * RT);
    int g, begin, end;
    if (!find_rows(a, slot, TOKENS, g, begin, end)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
    const int tokens = min(end - begin, TOKENS);
    const float ts = scale_of_sum(a.w_ts[g * a.w_ts_step], a.K);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // scalar bases, and offsets of 32 bits: K and ldx are below 2^24
    const uint32_t K = (uint32_t)a.K;
    const int rows = (int)min(a.N - n0, (int64_t)(16 * RT));
    const uint8_t* codes = a.w_codes + (g * a.N + n0) * (a.K / 2);
    const uint8_t* scales = a.w_scales + (g * a.N + n0) * (a.K / 16);
    const uint16_t* x = a.x + begin * a.ldx;
    uint32_t row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = (uint32_t)min(16 * i + r, rows - 1);

    f32x4_t acc[RT][TT], total[LONG ? RT : 1][LONG ? TT : 1];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            acc[i][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (LONG) total[i][t] = acc[i][t];
        }

    // load i brings tokens 4 i .. 4 i + 3; places of tokens that are not there
    // repeat the last one, units past K the last one of the row
    uint8_t* xs = smem + wave * (TOKENS * kUnits * 16);
    const uint32_t xs_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)xs;
    const uint32_t lt = lane >> 4, lu = lane & 15;
    auto load_tokens = [&](uint32_t k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TOKENS / 4; ++i) {
            const uint32_t t = 4 * i + lt;
            uint32_t k = k0 + 8 * (lu ^ (t & 15));
            if (!WHOLE) k = min(k, K - 8);
            load_to_lds(x, 2 * (min(t, (uint32_t)tokens - 1) * (uint32_t)a.ldx + k), xs_at + 1024 * i);
        }
    };
    // this wave's steps are [first, first + n): neighbouring steps share lines
    const uint32_t steps = (K + kStep - 1) / kStep, per_wave = (steps + WAVES - 1) / WAVES;
    const uint32_t first = min(wave * per_wave, steps), n = min(per_wave, steps - first);
    Codes w[RT];
    if (n > 0) {
        load_tokens(first * kStep);
#pragma unroll
        for (int i = 0; i < RT; ++i)
            load_codes(w[i], codes, scales, row[i], K, first * kStep + 32 * q, WHOLE || (first + 1) * kStep <= K);
    }
    for (uint32_t j = 0; j < n; ++j) {
        const uint32_t k0 = (first + j) * kStep;
        loads_done();
        bf16x8_t xf[TT][4];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int rt = TOKENS < 16 ? r % TOKENS : r;  // columns without a token repeat others
                u32x4 v = *reinterpret_cast<const u32x4*>(xs + ((16 * t + rt) * kUnits + ((4 * q + u) ^ rt)) * 16);
                if (!WHOLE && k0 + 32 * q + 8 * u >= K) v = u32x4{0u, 0u, 0u, 0u};
                __builtin_memcpy(&xf[t][u], &v, 16);
            }
        // The codes are in their registers; said here, so that the compiler does not
        // wait for the tokens below when it wants them.
#pragma unroll
        for (int i = 0; i < RT; ++i) asm volatile("" : "+v"(w[i].w), "+v"(w[i].s));
        const bool more = j + 1 < n;
        lds_reads_done();
        if (more) load_tokens(k0 + kStep);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float s0 = scale_value(w[i].s, 0), s1 = scale_value(w[i].s, 1);
            if (__builtin_expect(__any(any_nan(w[i].s)), 0)) {
                if ((w[i].s & 0xFFu) == kUe5m3Nan) s0 = __uint_as_float(0x7FC00000u);
                if ((w[i].s >> 8) == kUe5m3Nan) s1 = __uint_as_float(0x7FC00000u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bf16x8_t wv = dequant8(w[i].w[u], u < 2 ? s0 : s1);
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xf[t][u], acc[i][t], 0, 0, 0);
            }
            // the next codes into the registers that are free now
            if (more) load_codes(w[i], codes, scales, row[i], K, k0 + kStep + 32 * q, WHOLE || k0 + 2 * kStep <= K);
        }
        if constexpr (LONG)
            if (j % kFold == kFold - 1 || !more)
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            float s = total[i][t][d];
                            const float lost = fold(s, acc[i][t][d]);
                            total[i][t][d] = s;
                            acc[i][t][d] = more ? lost : s;
                        }
    }

    // ---- join the waves' sums: lane (r, q) holds rows 4 q .. 4 q + 3 of W for token r
    __syncthreads();
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(smem);  // [wave][RT][TT][lane]
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) sums[((wave * RT + i) * TT + t) * 64 + lane] = acc[i][t];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * TT * 64; e += 64 * WAVES) {
        const int l = e & 63, t = e / 64 % TT, i = e / 64 / TT;
        if (16 * t + (l & 15) >= tokens) continue;
        f32x4_t v = sums[e];
#pragma unroll
        for (int o = 1; o < WAVES; ++o) v += sums[o * (RT * TT * 64) + e];
        const int64_t to = (int64_t)begin + 16 * t + (l & 15), col = n0 + 16 * i + 4 * (l >> 4);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (col + d < a.N) {
                if (a.out_bf16) ((uint16_t*)a.out)[to * a.ldo + col + d] = to_bf16(v[d] * ts);
                else ((float*)a.out)[to * a.ldo + col + d] = v[d] * ts;
            }
        }
    }
}

// 32 codes of each of a chunk's 4 steps of 128 in row r, and the scale bytes of
// step q (8 of them) for lane q of the row's four.
struct ChunkCodes {
    u32x4 w[4];
    u32x2 s;
};
__device__ __forceinline__ void load_chunk(ChunkCodes& c, const uint8_t* codes, const uint8_t* scales, uint32_t row,
                                           uint32_t K, uint32_t k0, int q, bool whole) {
    if (__builtin_expect(whole, 1)) {
        const uint32_t at = row * (K / 2) + k0 / 2;
#pragma unroll
        for (int s = 0; s < 4; ++s) c.w[s] = *reinterpret_cast<const u32x4_at8*>(codes + at + 64 * s + 16 * q);
        c.s = *reinterpret_cast<const u32x2_at1*>(scales + (at >> 3) + 8 * q);
        return;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t at = row * (K / 16) + min(k0 + 128 * s + 32 * q + 16 * b, K - 16) / 16;
            const u32x2 v = *reinterpret_cast<const u32x2*>(codes + at * 8);
            c.w[s][2 * b] = v.x;
            c.w[s][2 * b + 1] = v.y;
        }
    }
    c.s = u32x2{0u, 0u};
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint32_t k = k0 + 128 * q + 16 * b;
        const uint32_t v = scales[row * (K / 16) + min(k, K - 16) / 16];
        c.s[b >> 2] |= (k < K ? v : 0u) << (8 * (b & 3));
    }
}

// The four lanes of a row hold 8 scale bytes each, lane s those of step s; lane q
// gets bytes 2 q and 2 q + 1 of each: steps 0 and 1 in the result's x, 2 and 3 in y.
// `pick` chooses the pair's half by q's low bit.
__device__ __forceinline__ u32x2 dealt(u32x2 s, uint32_t pick) {
    const auto a = __builtin_amdgcn_permlane32_swap(s.x, s.y, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
    return u32x2{__builtin_amdgcn_perm(b[1], b[0], pick), __builtin_amdgcn_perm(c[1], c[0], pick)};
}

// The same in chunks of 4 steps: fewer loads of scales, and all of a chunk's codes
// are on their way at once.  The tokens of PART steps stand in LDS; they are read
// into registers before the next ones are asked for, or (4 tokens) have two places.
// 16 tokens, 16384 -> 4096: 16.7 us (2.3 TB/s), in steps of 128 it took 32 us; the bytes
// alone would take 7.5.  With RT = 1 a wave asks for its next chunk behind its last
// product and then waits for all loads, so it has no weights in flight while it
// multiplies, and a CU has two such waves per SIMD.
template <int RT, int TOKENS, int WAVES, bool WHOLE>
__global__ __launch_bounds__(64 * WAVES, RT > 2 ? 2 : RT * TOKENS >= 32 ? 3 : 4) void chunks_kernel(WeightOnlyArgs a, Place place) {
    constexpr int kChunk = 512, PART = TOKENS > 4 ? 2 : 4, kPlaces = TOKENS > 4 ? 1 : 2;
    static_assert(TOKENS <= 16, "one tile of tokens");
    constexpr int kStepBytes = TOKENS * 256, kWaveBytes = kPlaces * PART * kStepBytes;
    constexpr int kTokenBytes = WAVES * kWaveBytes, kSumBytes = WAVES * RT * 64 * 16;
    __shared__ __align__(16) uint8_t smem[kTokenBytes > kSumBytes ? kTokenBytes : kSumBytes];
    const uint32_t u0 = place.tile + blockIdx.x, down = u0 / place.tiles;
    const int64_t slot = place.slot + down, n0 = (int64_t)(u0 - down * place.tiles) * (16 * RT);
    int g, begin, end;
    if (!find_rows(a, slot, TOKENS, g, begin, end)) return;
    g = __builtin_amdgcn_readfirstlane(g);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
    const int tokens = min(end - begin, TOKENS);
    const float ts = scale_of_sum(a.w_ts[g * a.w_ts_step], a.K);
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t K = (uint32_t)a.K;
    const int rows = (int)min(a.N - n0, (int64_t)(16 * RT));
    const uint8_t* codes = a.w_codes + (g * a.N + n0) * (a.K / 2);
    const uint8_t* scales = a.w_scales + (g * a.N + n0) * (a.K / 16);
    const uint16_t* x = a.x + begin * a.ldx;
    const uint32_t pick = q & 1 ? 0x07060302u : 0x05040100u;
    uint32_t row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = (uint32_t)min(16 * i + r, rows - 1);
    f32x4_t acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    uint8_t* xs = smem + wave * kWaveBytes;
    const uint32_t xs_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)xs;
    const uint32_t lt = lane >> 4, lu = lane & 15;
    auto load_tokens = [&](uint32_t k0, uint32_t at) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < PART; ++s)
#pragma unroll
            for (int i = 0; i < TOKENS / 4; ++i) {
                const uint32_t t = 4 * i + lt;
                uint32_t k = k0 + 128 * s + 8 * (lu ^ (t & 15));
                if (!WHOLE) k = min(k, K - 8);
                load_to_lds(x, 2 * (min(t, (uint32_t)tokens - 1) * (uint32_t)a.ldx + k), at + s * kStepBytes + 1024 * i);
            }
    };
    // chunk j of this wave is chunk wave + WAVES j of K
    const uint32_t first = wave * kChunk, stride = WAVES * kChunk;
    ChunkCodes w[RT];
    if (first < K) {
        load_tokens(first, xs_at);
#pragma unroll
        for (int i = 0; i < RT; ++i) load_chunk(w[i], codes, scales, row[i], K, first, q, WHOLE || first + kChunk <= K);
    }
    uint32_t at = 0;  // the place that holds the tokens
    for (uint32_t k0 = first; k0 < K; k0 += stride) {
        const uint32_t next = k0 + stride;
        u32x2 sc[RT];
        bool nan = false;
#pragma unroll
        for (int part = 0; part < 4 / PART; ++part) {
            loads_done();
            if (part == 0) {
                // The codes are in their registers; said here, so that the compiler
                // does not wait for the next tokens when it wants them.
                uint32_t bad = 0u;
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    asm volatile("" : "+v"(w[i].w[0]), "+v"(w[i].w[1]), "+v"(w[i].w[2]), "+v"(w[i].w[3]), "+v"(w[i].s));
                    bad |= any_nan(w[i].s.x) | any_nan(w[i].s.y);
                    sc[i] = dealt(w[i].s, pick);
                }
                nan = __any(bad);
            }
            const uint8_t* from = xs + at * (PART * kStepBytes);
            auto fragment = [&](int s, int u) __attribute__((always_inline)) {
                const int rt = TOKENS < 16 ? r % TOKENS : r;  // columns without a token repeat others
                u32x4 v = *reinterpret_cast<const u32x4*>(from + s * kStepBytes + (rt * 16 + ((4 * q + u) ^ rt)) * 16);
                if (!WHOLE && k0 + 128 * (PART * part + s) + 32 * q + 8 * u >= K) v = u32x4{0u, 0u, 0u, 0u};
                bf16x8_t o;
                __builtin_memcpy(&o, &v, 16);
                return o;
            };
            bf16x8_t xf[PART][4];
            if (kPlaces == 1) {
#pragma unroll
                for (int s = 0; s < PART; ++s)
#pragma unroll
                    for (int u = 0; u < 4; ++u) xf[s][u] = fragment(s, u);
            }
            lds_reads_done();  // of the place that is loaded next: just now, or (two places) a turn ago
            const bool last = part == 4 / PART - 1;
            const uint32_t kx = last ? next : k0 + 128 * PART * (part + 1);
            if (kx < K) load_tokens(kx, xs_at + (kPlaces - 1) * (at ^ 1) * (PART * kStepBytes));
#pragma unroll
            for (int i = 0; i < RT; ++i) {
#pragma unroll
                for (int s = 0; s < PART; ++s) {
                    const int step = PART * part + s;
                    const uint32_t two = (step < 2 ? sc[i].x : sc[i].y) >> (16 * (step & 1));
                    float s0 = scale_value(two, 0), s1 = scale_value(two, 1);
                    if (__builtin_expect(nan, 0)) {
                        if ((two & 0xFFu) == kUe5m3Nan) s0 = __uint_as_float(0x7FC00000u);
                        if (((two >> 8) & 0xFFu) == kUe5m3Nan) s1 = __uint_as_float(0x7FC00000u);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const bf16x8_t xu = kPlaces == 1 ? xf[s][u] : fragment(s, u);
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dequant8(w[i].w[step][u], u < 2 ? s0 : s1), xu, acc[i], 0, 0, 0);
                    }
                }
                // the next codes into the registers that are free now
                if (last && next < K) load_chunk(w[i], codes, scales, row[i], K, next, q, WHOLE || next + kChunk <= K);
            }
            if (kPlaces == 2) at ^= 1;
            if (!WHOLE && !last && kx >= K) break;  // the chunk ends before its second half: it is the last
        }
    }

    // ---- join the waves' sums: lane (r, q) holds rows 4 q .. 4 q + 3 of W for token r
    __syncthreads();
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(smem);  // [wave][RT][lane]
#pragma unroll
    for (int i = 0; i < RT; ++i) sums[(wave * RT + i) * 64 + lane] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * 64; e += 64 * WAVES) {
        const int l = e & 63, i = e / 64;
        if ((l & 15) >= tokens) continue;
        f32x4_t v = sums[e];
#pragma unroll
        for (int o = 1; o < WAVES; ++o) v += sums[o * (RT * 64) + e];
        const int64_t to = (int64_t)begin + (l & 15), col = n0 + 16 * i + 4 * (l >> 4);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if (col + d < a.N) {
                if (a.out_bf16) ((uint16_t*)a.out)[to * a.ldo + col + d] = to_bf16(v[d] * ts);
                else ((float*)a.out)[to * a.ldo + col + d] = v[d] * ts;
            }
        }
    }
}

template <int ROWS, int WAVES, bool LONG = false>
void launch_one(const WeightOnlyArgs& a, hipStream_t stream) {
    const int64_t tiles_n = (a.N + ROWS - 1) / ROWS;
    in_launches(a.rows * tiles_n, 64 * WAVES, [&](int64_t first, dim3 grid) {
        const Place at{first / tiles_n, (uint32_t)(first % tiles_n), (uint32_t)tiles_n};
        if (!LONG && a.K % 512 == 0) hipLaunchKernelGGL((one_token_kernel<ROWS, WAVES, true, false>), grid, dim3(64 * WAVES), 0, stream, a, at);
        else hipLaunchKernelGGL((one_token_kernel<ROWS, WAVES, false, LONG>), grid, dim3(64 * WAVES), 0, stream, a, at);
    });
}

template <int RT, int TOKENS, int WAVES>
void launch_chunks(const WeightOnlyArgs& a, hipStream_t stream) {
    const int64_t tiles_n = (a.N + 16 * RT - 1) / (16 * RT);
    int64_t slots = (a.rows + TOKENS - 1) / TOKENS;
    if (a.offsets) slots = a.rows / TOKENS + (a.experts < a.rows ? a.experts : a.rows);
    in_launches(slots * tiles_n, 64 * WAVES, [&](int64_t first, dim3 grid) {
        const Place at{first / tiles_n, (uint32_t)(first % tiles_n), (uint32_t)tiles_n};
        if (a.K % 512 == 0) hipLaunchKernelGGL((chunks_kernel<RT, TOKENS, WAVES, true>), grid, dim3(64 * WAVES), 0, stream, a, at);
        else hipLaunchKernelGGL((chunks_kernel<RT, TOKENS, WAVES, false>), grid, dim3(64 * WAVES), 0, stream, a, at);
    });
}

template <int RT, int TOKENS, int WAVES, bool LONG = false>
void launch(const WeightOnlyArgs& a, hipStream_t stream) {
    const int64_t tiles_n = (a.N + 16 * RT - 1) / (16 * RT);
    int64_t slots = (a.rows + TOKENS - 1) / TOKENS;
    if (a.offsets) slots = a.rows / TOKENS + (a.experts < a.rows ? a.experts : a.rows);
    in_launches(slots * tiles_n, 64 * WAVES, [&](int64_t first, dim3 grid) {
        const Place at{first / tiles_n, (uint32_t)(first % tiles_n), (uint32_t)tiles_n};
        if (!LONG && a.K % 128 == 0) hipLaunchKernelGGL((tokens_kernel<RT, TOKENS, WAVES, true, false>), grid, dim3(64 * WAVES), 0, stream, a, at);
        else hipLaunchKernelGGL((tokens_kernel<RT, TOKENS, WAVES, false, LONG>), grid, dim3(64 * WAVES), 0, stream, a, at);
    });
}

}  // namespace

// What a workgroup has.  Rows of W: joining 32 or 64 halves the reads of the tokens, and
// workgroups.  Waves, which share out K: 8 have the most loads in flight where there are
// few workgroups (16384 -> 4096, 4 tokens, 12.7 us, with 4 waves 16.5); where there are
// many, fewer leave none idle when K is short and join fewer sums.  Experts, us:
//   1 token    16 of 64 experts 1024 -> 4096  16 rows, 8 waves 21.1   16, 2  10.8   16, 4  13.1
//   16 tokens  9 experts 2064 -> 1305         32, 8  12.8             16, 4   9.0
//              64 experts 4096 -> 2048        64, 8  92.6             32, 4  68.0
//              64 experts 1024 -> 4096        16, 8 131               64, 2  43.9   32, 4  50.4
//   64 tokens  64 experts 1024 -> 4096        16, 8 280               32, 2  96.4   32, 4 110
// One matrix, on both sides of the borders below, us (workgroups that 16 rows each make):
//                        256    384    512    768   1024   1536   2048   4096
//   1 token   16, 8                    6.1    8.6    9.8   13.6   17.2   31.5   K = 4096
//             16, 4                    6.0    7.6    8.7   11.7   14.9   26.8
//             16, 8                    9.7   14.5   16.4   23.1   29.4   54.5   K = 8192
//             16, 4                   10.4   13.9   17.1   24.5   30.8   56.9
//             16, 4                    3.9    4.1    4.5    6.1    7.0   10.9   K = 1024
//             16, 2                    3.9    4.2    4.3    5.6    6.1    9.0
//             16, 4                    4.2    4.7    5.4    7.0    8.2   12.8   K = 1536
//             16, 2                    4.4    4.8    5.6    6.9    7.9   13.1
//   4 tokens  16, 8      5.5    7.7    8.0   10.6   13.2   18.8   23.8   45.2   K = 4096
//             16, 4      6.1    7.8    8.0   10.5   12.0   16.9   20.6   36.4
//             32, 4      8.2    8.9    9.3   11.6   12.0   16.4   19.5   33.7
//             32, 4                                  6.8    7.7    8.6   14.3   K = 1024
//             32, 2                                  6.7    7.9    8.3   11.5
//   16 tokens 16, 8      6.2    9.8   10.1   14.0   17.1   23.9   30.3   56.7   K = 4096
//             16, 4      6.5    9.4    9.7   13.3   16.2   22.9   28.6   53.1
//             32, 4      8.3    9.4   10.0   13.8   14.4   19.0   23.7   44.4
//             32, 4                                  6.7    8.0    9.1   15.4   K = 1024
//             64, 2                                  7.5   10.6   10.9   14.3
//   32 tokens 16, 8      7.2   13.9   14.3   19.9   25.2   36.6   47.3   90.3   K = 4096
//             32, 4     10.2   12.2   12.8   19.5   20.1   28.7   37.1   70.4
//   64 tokens 16, 8     10.0   20.0   20.9   29.7   38.3   56.4   74.0  145     K = 4096
//             32, 4     12.8   14.8   15.7   26.1   26.4   38.2   48.6   91.5
//             32, 4                    6.7    9.0    9.1   14.6   17.1   31.0   K = 1024
//             32, 2                    8.4    9.8   10.0   13.4   16.1   31.6
// The forms cross where the rule changes or are within a tenth of each other there, but
// for 8 waves kept from 512 to 1024 (1 token) and from 256 to 512 (32 and 64
// tokens), which cost up to a third there, and 64 rows at 2048 of K = 1024, a fifth.
void launch_gemm_weight_only(const WeightOnlyArgs& a, hipStream_t stream) {
    // Tokens that a workgroup should be ready for: all, or of an expert twice the
    // mean (more than that take the weights a second time).
    const int64_t each = !a.offsets ? a.rows : a.rows <= a.experts / 4 ? 1 : 2 * ((a.rows + a.experts - 1) / a.experts);
    // Workgroups that 16 rows of W each would make.
    const int64_t blocks = a.offsets ? (a.experts < a.rows ? a.experts : a.rows) : (a.rows + 63) / 64;
    const int64_t groups = (a.N + 15) / 16 * blocks;
    if (a.K > kChain) {
        if (each == 1) launch_one<16, 8, true>(a, stream);
        else if (each <= 16) launch<1, 16, 8, true>(a, stream);
        else launch<1, 64, 8, true>(a, stream);
    } else if (each == 1) {
        if (groups >= 2048 && a.K <= 1024) launch_one<16, 2>(a, stream);
        else if (groups >= 1024 && a.K <= 5120) launch_one<16, 4>(a, stream);
        else launch_one<16, 8>(a, stream);
    } else if (each <= 4) {
        if (groups < 512) launch_chunks<1, 4, 8>(a, stream);
        else if (groups < 2048) launch_chunks<1, 4, 4>(a, stream);
        else if (a.K <= 1024) launch_chunks<2, 4, 2>(a, stream);
        else launch_chunks<2, 4, 4>(a, stream);
    } else if (each <= 16) {
        if (groups < 512) launch_chunks<1, 16, 8>(a, stream);
        else if (groups < 1024) launch_chunks<1, 16, 4>(a, stream);
        else if (groups >= 2048 && a.K <= 1024) launch_chunks<4, 16, 2>(a, stream);
        else launch_chunks<2, 16, 4>(a, stream);
    } else if (each <= 32) {
        if (groups < 512) launch<1, 32, 8>(a, stream);
        else if (groups >= 4096 && a.K <= 1024) launch<2, 32, 2>(a, stream);
        else launch<2, 32, 4>(a, stream);
    } else {
        if (groups < 512) launch<1, 64, 8>(a, stream);
        else if (groups >= 4096 && a.K <= 1024) launch<2, 64, 2>(a, stream);
        else launch<2, 64, 4>(a, stream);
    }
}

}  // namespace ue5m3fp4
