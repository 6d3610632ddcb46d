// Dropout from the counter-based generator, fused with the residual addition
// and the tensor amax; forward and backward are the same pass (the mask is
// drawn again from the counters, never stored).  Arithmetic and counter
// layout: include/ue5m3fp4_layer.h; Philox4x32-10: formats.hpp.
//
// One Philox call serves 8 consecutive elements (16 bits each), which is the
// unit a thread loads (16 bytes of bf16), draws for and stores.  A thread takes 4
// units a workgroup apart; in small tensors, which would leave CUs idle, 1.
//
// Bound: HBM, with the generator's arithmetic hidden under it (vector ALU busy
// 0.28 to 0.59).  Measured on inputs rotated past the 256 MB cache: 8192 x 4096
// fp32 + bf16 residual -> bf16 with the amax 46 us (5.8 TB/s), backward of 8192 x
// 16384 bf16 92 us (5.8 TB/s); a plain copy runs at 5.1 to 5.5 on the same card.
// Rows that do not start at whole units (an odd row stride, or odd columns in
// wider rows) go element by element: 8192 x 4096 bf16 92 us, against 26.
#include "../formats.hpp"
#include "layer.hpp"

namespace ue5m3fp4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kSmall = 256 * 2048;  // units that still fit one per thread of 256 CUs
constexpr uint32_t kStream = 2; // third counter word: dropout's own stream

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};  // round to nearest even
    return __builtin_bit_cast(uint32_t, v);
}

// 8 consecutive elements as fp32, 16-byte aligned.
template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t off, float (&v)[8]) {
    if constexpr (F32) {
        const f32x4* p = reinterpret_cast<const f32x4*>((const float*)base + off);
        const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    } else {
        const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const uint16_t*)base + off));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[2 * e] = bf16_lo(w[e]), v[2 * e + 1] = bf16_hi(w[e]);
    }
}

template <bool F32>
__device__ __forceinline__ float load1(const void* base, int64_t off) {
    if constexpr (F32) return ((const float*)base)[off];
    else return __uint_as_float((uint32_t)((const uint16_t*)base)[off] << 16);
}

// The value kept by out's type, as fp32 bits without the sign (orders as the
// magnitude, NaN above Inf).
template <bool F32>
__device__ __forceinline__ uint32_t store8(void* base, int64_t off, const float (&v)[8]) {
    uint32_t m = 0u;
    if constexpr (F32) {
        f32x4* p = reinterpret_cast<f32x4*>((float*)base + off);
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    } else {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            m = max(m, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
        }
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>((uint16_t*)base + off));
    }
    return m;
}

template <bool F32>
__device__ __forceinline__ uint32_t store1(void* base, int64_t off, float v) {
    if constexpr (F32) {
        ((float*)base)[off] = v;
        return __float_as_uint(v) & 0x7FFFFFFFu;
    } else {
        const uint32_t w = pack_bf16(v, 0.0f) & 0xFFFFu;
        ((uint16_t*)base)[off] = (uint16_t)w;
        return (w << 16) & 0x7FFFFFFFu;
    }
}

// Workgroup maximum of m folded into *amax: one atomic, skipped when the
// running value is already as large (it only grows).
__device__ __forceinline__ void amax_commit32(uint32_t m, float* amax) {
    __shared__ uint32_t wave_max[kThreads / 64];
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 64; ++i) m = max(m, wave_max[i]);
        unsigned int* dst = reinterpret_cast<unsigned int*>(amax);
        if (m > __hip_atomic_load(dst, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(dst, m);
    }
}

// VEC: units of 8 elements are 16-byte aligned in every tensor and lie in one
// row (contiguous tensors are passed as a single row; the last, partial unit
// of one goes element by element).  W32: every call number fits 32 bits.
template <bool XF32, bool OF32, bool RES, bool VEC, bool W32, int kUnits>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutArgs a) {
    const int64_t n = a.rows * a.cols, units = (n + 7) / 8;
    const int64_t u0 = (blockIdx.x + a.first) * (kThreads * kUnits) + threadIdx.x;
    uint32_t m = 0u;
    auto words = [&](int64_t u) __attribute__((always_inline)) {
        if constexpr (W32) return sr_words32((uint32_t)u, a.offset, kStream, a.seed);
        else return sr_words((uint64_t)u, a.offset, kStream, a.seed);
    };
    auto drop = [&](float x, uint32_t u16) __attribute__((always_inline)) {
        return u16 >= a.threshold ? x * a.scale : 0.0f;
    };
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int64_t u = u0 + k * kThreads;
        if (u >= units) break;
        const int64_t e0 = u * 8;
        int64_t row = 0, col = e0;
        if (a.rows > 1) {
            row = e0 / a.cols;
            col = e0 - row * a.cols;
        }
        const U32x4 w = words(u);
        if (VEC && e0 + 8 <= n) {
            float v[8];
            load8<XF32>(a.x, row * a.ldx + col, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = drop(v[e], sr_u16(w, e));
            if constexpr (RES) {
                float r[8];
                load8<OF32>(a.residual, row * a.ldr + col, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = r[e] + v[e];
            }
            m = max(m, store8<OF32>(a.out, row * a.ldo + col, v));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e0 + e < n) {
                    float v = drop(load1<XF32>(a.x, row * a.ldx + col), sr_u16(w, e));
                    if constexpr (RES) v = load1<OF32>(a.residual, row * a.ldr + col) + v;
                    m = max(m, store1<OF32>(a.out, row * a.ldo + col, v));
                    if (++col == a.cols) {
                        col = 0;
                        ++row;
                    }
                }
            }
        }
    }
    if (a.amax != nullptr) amax_commit32(m, a.amax);
}

template <bool XF32, bool OF32, bool RES, bool VEC, bool W32, int kUnits>
void launch_units(const DropoutArgs& a, int64_t units, hipStream_t stream) {
    in_launches((units + kThreads * kUnits - 1) / (kThreads * kUnits), kThreads, [&](int64_t first, dim3 grid) {
        DropoutArgs part = a;
        part.first = first;
        hipLaunchKernelGGL((dropout_kernel<XF32, OF32, RES, VEC, W32, kUnits>), grid, dim3(kThreads), 0, stream, part);
    });
}

template <bool XF32, bool OF32, bool RES, bool VEC>
void launch_w(const DropoutArgs& a, hipStream_t stream) {
    const int64_t units = (a.rows * a.cols + 7) / 8;
    if (units <= kSmall) launch_units<XF32, OF32, RES, VEC, true, 1>(a, units, stream);
    else if (units <= ((int64_t)1 << 32)) launch_units<XF32, OF32, RES, VEC, true, 4>(a, units, stream);
    else launch_units<XF32, OF32, RES, VEC, false, 4>(a, units, stream);
}

template <bool XF32, bool OF32, bool RES>
void launch_v(const DropoutArgs& a, bool vec, hipStream_t stream) {
    vec ? launch_w<XF32, OF32, RES, true>(a, stream) : launch_w<XF32, OF32, RES, false>(a, stream);
}

template <bool XF32, bool OF32>
void launch_r(const DropoutArgs& a, bool vec, hipStream_t stream) {
    a.residual ? launch_v<XF32, OF32, true>(a, vec, stream) : launch_v<XF32, OF32, false>(a, vec, stream);
}

}  // namespace

void launch_dropout(const DropoutArgs& args, hipStream_t stream) {
    DropoutArgs a = args;
    if (!a.residual) a.ldr = a.ldx;
    bool vec = a.cols % 8 == 0 && a.ldx % 8 == 0 && a.ldo % 8 == 0 && a.ldr % 8 == 0;
    if (a.rows == 1 || (a.ldx == a.cols && a.ldo == a.cols && (!a.residual || a.ldr == a.cols))) {
        a.cols *= a.rows;  // contiguous: one row of rows x cols elements
        a.rows = 1;
        vec = true;
    }
    if (a.x_f32) a.out_f32 ? launch_r<true, true>(a, vec, stream) : launch_r<true, false>(a, vec, stream);
    else a.out_f32 ? launch_r<false, true>(a, vec, stream) : launch_r<false, false>(a, vec, stream);
}

}  // namespace ue5m3fp4
