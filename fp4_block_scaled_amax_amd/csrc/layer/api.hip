// C ABI of libue5m3fp4_layer (declared in include/ue5m3fp4_layer.h): argument
// checks on the host, then one launch on the caller's stream.  No allocation,
// no synchronization, no retained state.
#include <cmath>

#include "../../../include/ue5m3fp4_layer.h"
#include "layer.hpp"

namespace {

using namespace ue5m3fp4;

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxFp8K = (int64_t)1 << 24;  // a GEMM tile's code offsets fit 32 bits

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool is01(int v) { return v == 0 || v == 1; }

// rows x ld elements, checked without a product that could wrap
bool too_large(int64_t rows, int64_t ld) { return ld >= kMaxElems || (ld > 0 && rows > (kMaxElems - 1) / ld); }

// The runtime's per-thread last-error slot may hold an earlier, unrelated
// error: it is cleared right before the launches, so that launch_status
// reports only their own failures.
void clear_stale_error() { (void)hipGetLastError(); }

int launch_status() { return hipGetLastError() == hipSuccess ? UE5M3FP4_OK : UE5M3FP4_EHIP; }

int run_dropout(const void* x, int x_type, int64_t ldx, const void* residual, int64_t ldr, void* out, int out_type,
                int64_t ldo, int64_t rows, int64_t cols, double p, uint64_t seed, uint32_t offset, float* amax,
                void* stream) {
    if (rows < 0 || cols < 0 || ldx < 0 || ldo < 0 || !is01(x_type) || !is01(out_type)) return UE5M3FP4_EINVAL;
    if (!(p >= 0.0 && p <= 1.0)) return UE5M3FP4_EINVAL;
    if (!residual) ldr = cols;
    if (ldr < 0) return UE5M3FP4_EINVAL;
    // cols only by rows * ld: a contiguous tensor of any shape is one row
    if (rows >= kMaxDim || cols >= kMaxElems || too_large(rows, ldx) || too_large(rows, ldo) || too_large(rows, ldr))
        return UE5M3FP4_ERANGE;
    if (rows == 0 || cols == 0) return UE5M3FP4_OK;
    if (!x || !out) return UE5M3FP4_EINVAL;
    if (ldx < cols || ldo < cols || ldr < cols) return UE5M3FP4_ESHAPE;
    if (!aligned16(x) || !aligned16(out) || (residual && !aligned16(residual)) || (amax && !aligned4(amax)))
        return UE5M3FP4_EALIGN;
    const uint32_t t = (uint32_t)std::nearbyint(65536.0 * p);
    const float scale = t == 65536u ? 0.0f : (float)(65536.0 / (65536.0 - (double)t));
    const DropoutArgs a{x,    residual, out,  x_type == UE5M3FP4_F32, out_type == UE5M3FP4_F32, ldx, ldr, ldo,
                        rows, cols,     t,    scale,                  seed,                     offset, amax, 0};
    clear_stale_error();
    launch_dropout(a, (hipStream_t)stream);
    return launch_status();
}

}  // namespace

extern "C" {

int ue5m3fp4_quantize_fp8(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int format, int scale_type,
                          int tile, uint8_t* row_codes, void* row_scales, uint8_t* col_codes, void* col_scales,
                          void* stream) {
    if (rows < 0 || cols < 0 || ld < 0 || !is01(format) || !is01(scale_type) || !is01(tile)) return UE5M3FP4_EINVAL;
    if (rows >= kMaxDim || cols >= kMaxDim || too_large(rows, ld)) return UE5M3FP4_ERANGE;
    if (rows == 0 || cols == 0) return UE5M3FP4_OK;  // empty tensor: nothing to do
    if (!x) return UE5M3FP4_EINVAL;
    if ((row_codes == nullptr) != (row_scales == nullptr) || (col_codes == nullptr) != (col_scales == nullptr))
        return UE5M3FP4_EINVAL;
    if (!row_codes && !col_codes) return UE5M3FP4_EINVAL;  // no output requested
    if (row_codes == col_codes || row_scales == col_scales) return UE5M3FP4_EINVAL;  // one buffer for both
    if (ld < cols) return UE5M3FP4_ESHAPE;
    if (!aligned16(x) || !aligned16(row_codes) || !aligned16(row_scales) || !aligned16(col_codes) ||
        !aligned16(col_scales))
        return UE5M3FP4_EALIGN;
    const QuantizeFp8Args a{x,    rows,      cols,       ld,        format == UE5M3FP4_E5M2, scale_type == UE5M3FP4_SCALE_E8M0,
                            tile == 1, row_codes, row_scales, col_codes, col_scales, 0};
    clear_stale_error();
    launch_quantize_fp8(a, (hipStream_t)stream);
    return launch_status();
}

int ue5m3fp4_gemm_fp8_nt(const uint8_t* a_codes, const void* a_scales, int a_format, int a_tile,
                         const uint8_t* b_codes, const void* b_scales, int b_format, int b_tile, int scale_type,
                         int64_t M, int64_t N, int64_t K, void* c, int c_type, void* stream) {
    if (M < 0 || N < 0 || K < 0 || !is01(a_format) || !is01(b_format) || !is01(a_tile) || !is01(b_tile) ||
        !is01(scale_type) || !is01(c_type))
        return UE5M3FP4_EINVAL;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxFp8K) return UE5M3FP4_ERANGE;
    const int64_t Kp = (K + 127) / 128 * 128;
    if (M * N >= kMaxElems || M * Kp >= kMaxElems || N * Kp >= kMaxElems) return UE5M3FP4_ERANGE;
    if (M == 0 || N == 0) return UE5M3FP4_OK;  // nothing is read or written
    if (!c) return UE5M3FP4_EINVAL;
    if (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return UE5M3FP4_EINVAL;
    if (!aligned16(c)) return UE5M3FP4_EALIGN;
    if (K > 0 && (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales)))
        return UE5M3FP4_EALIGN;
    const GemmFp8Args g{{a_codes, a_scales, a_format == UE5M3FP4_E5M2, a_tile == 1},
                        {b_codes, b_scales, b_format == UE5M3FP4_E5M2, b_tile == 1},
                        scale_type == UE5M3FP4_SCALE_E8M0, M, N, K, c, c_type == UE5M3FP4_BF16, 0};
    clear_stale_error();
    launch_gemm_fp8(g, (hipStream_t)stream);
    return launch_status();
}

int ue5m3fp4_dropout(const void* x, int x_type, int64_t ldx, const void* residual, int64_t ldr, void* out,
                     int out_type, int64_t ldo, int64_t rows, int64_t cols, double p, uint64_t seed, uint32_t offset,
                     float* amax_inout, void* stream) {
    return run_dropout(x, x_type, ldx, residual, ldr, out, out_type, ldo, rows, cols, p, seed, offset, amax_inout,
                       stream);
}

int ue5m3fp4_dropout_backward(const void* dy, int dy_type, int64_t lddy, void* dx, int dx_type, int64_t lddx,
                              int64_t rows, int64_t cols, double p, uint64_t seed, uint32_t offset,
                              float* amax_inout, void* stream) {
    return run_dropout(dy, dy_type, lddy, nullptr, 0, dx, dx_type, lddx, rows, cols, p, seed, offset, amax_inout,
                       stream);
}

}  // extern "C"
