// Internal launch interface between the C ABI (experts/api.hip) and the
// kernels, and what the kernels share.  Callers have validated every argument;
// launchers only enqueue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../layer/layer.hpp"  // in_launches

namespace ue5m3fp4 {

struct QuantizeGroupedArgs {
    const uint16_t* x;
    int64_t x_rows, cols, ld;
    const int32_t* index;  // nullable
    int64_t rows;
    const int32_t* offsets;
    int experts;
    const float* tensor_scale;
    bool stochastic;
    uint64_t seed;
    uint32_t offset;
    uint8_t* row_codes;  // nullable pairs
    uint8_t* row_scales;
    uint8_t* col_codes;
    uint8_t* col_scales;
    float* amax;  // nullable
};

void launch_quantize_grouped(const QuantizeGroupedArgs& a, hipStream_t stream);

struct GemmGroupedArgs {
    const uint8_t* a_codes;
    const uint8_t* a_scales;
    const float* a_ts;
    const uint8_t* b_codes;
    const uint8_t* b_scales;
    const float* b_ts;
    int64_t b_ts_step;  // 0: one tensor scale for all experts
    const int32_t* offsets;
    int experts;
    int64_t rows;     // grouped rows
    int64_t M, N, K;  // M: wgrad only; K: fprop and dgrad only
    void* c;
    bool c_bf16;
    float* amax;    // nullable
    int64_t first;  // the launch's first workgroup (set by the launcher)
};

void launch_gemm_grouped_nt(const GemmGroupedArgs& g, hipStream_t stream);
void launch_gemm_grouped_wgrad(const GemmGroupedArgs& g, hipStream_t stream);

struct WeightOnlyArgs {
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* w_codes;
    const uint8_t* w_scales;
    const float* w_ts;
    int64_t w_ts_step;
    const int32_t* offsets;  // null: one matrix
    int experts;
    int64_t rows, N, K;
    void* out;
    bool out_bf16;
    int64_t ldo;
};

void launch_gemm_weight_only(const WeightOnlyArgs& a, hipStream_t stream);

// Columns of a grouped transposed operand.
inline int64_t rows_padded(int64_t rows, int64_t experts) { return 128 * ((rows + 127) / 128 + experts); }

// ------------------------------------------------------------ device side --

// The rows of expert g, whatever the offsets hold: 0 <= begin <= end <= rows.
struct GroupRows {
    int begin, end;
};
__device__ __forceinline__ GroupRows group_rows(const int32_t* offsets, int g, int rows) {
    GroupRows r;
    r.begin = min(max(offsets[g], 0), rows);
    r.end = min(max(offsets[g + 1], r.begin), rows);
    return r;
}

// First column of expert g's rows in a grouped transposed operand.
__device__ __forceinline__ int64_t padded_begin(int begin, int g) {
    return 128 * (((int64_t)begin + 127) / 128 + g);
}

// The scale of a sum of K terms.  Of none it is 0 under any tensor scale, NaN and the
// infinities (which 0 times them would not be) among them.
__device__ __forceinline__ float scale_of_sum(float ts, int64_t K) { return K > 0 ? ts : __builtin_copysignf(1.0f, ts); }

// sum + part; returns what that rounds off, which belongs to the next part (nothing of an
// infinity or NaN).
__device__ __forceinline__ float fold(float& sum, float part) {
    const float s = sum + part, b = s - sum, lost = (sum - (s - b)) + (part - b);
    sum = s;
    return s - s == 0.0f ? lost : 0.0f;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(v, d);
        v += lane >= d ? o : 0;
    }
    return v;
}

}  // namespace ue5m3fp4
