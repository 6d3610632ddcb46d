// Internal launch interface between the C ABI (layer/api.hip) and the
// kernels.  Callers have validated every argument; launchers only enqueue.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ue5m3fp4 {

// A grid of any number of workgroups, as launches of at most 2^32 - 1 threads:
// beyond that HIP starts their number modulo 2^32, without an error.
// launch(first, grid) starts workgroups first .. first + grid - 1; first is a
// multiple of 8, so that the XCDs keep their turns.
template <typename F>
void in_launches(int64_t groups, int threads, F launch) {
    const int64_t most = 0xFFFFFFFFll / threads / 8 * 8;
    for (int64_t first = 0; first < groups; first += most) {
        const int64_t rest = groups - first;
        launch(first, dim3((unsigned)(rest < most ? rest : most)));
    }
}

struct QuantizeFp8Args {
    const uint16_t* x;
    int64_t rows, cols, ld;
    bool e5m2, e8m0, tile;
    uint8_t* row_codes;  // nullable pairs
    void* row_scales;
    uint8_t* col_codes;
    void* col_scales;
    int64_t first;  // the launch's first tile (set by the launcher)
};

void launch_quantize_fp8(const QuantizeFp8Args& a, hipStream_t stream);

struct Fp8Operand {
    const uint8_t* codes;  // [rows][K rounded up to 128]
    const void* scales;    // [blocks][rows] or, for tiles, [blocks][ceil(rows / 128)]
    bool e5m2, tile;
};

struct GemmFp8Args {
    Fp8Operand a, b;
    bool e8m0;
    int64_t M, N, K;
    void* c;
    bool c_bf16;
    int64_t first;  // the launch's first tile (set by the launcher)
};

void launch_gemm_fp8(const GemmFp8Args& g, hipStream_t stream);

struct DropoutArgs {
    const void* x;
    const void* residual;  // nullable
    void* out;
    bool x_f32, out_f32;
    int64_t ldx, ldr, ldo, rows, cols;
    uint32_t threshold;  // an element is kept iff its 16 bits are >= threshold
    float scale;
    uint64_t seed;
    uint32_t offset;
    float* amax;    // nullable
    int64_t first;  // the launch's first workgroup (set by the launcher)
};

void launch_dropout(const DropoutArgs& a, hipStream_t stream);

}  // namespace ue5m3fp4
