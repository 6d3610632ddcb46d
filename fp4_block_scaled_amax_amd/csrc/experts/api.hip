// C ABI of libue5m3fp4_experts (declared in include/ue5m3fp4_experts.h):
// argument checks on the host, then the launch on the caller's stream.  No
// allocation, no synchronization, no retained state.
#include "../../../include/ue5m3fp4_experts.h"
#include "experts.hpp"

namespace {

using namespace ue5m3fp4;

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxExperts = 65536;
constexpr int64_t kMaxK = (int64_t)1 << 24;  // of a product: offsets inside a tile fit 32 bits

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned8(const void* p) { return ((uintptr_t)p & 7u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool is01(int v) { return v == 0 || v == 1; }

// a x b elements (both non-negative), checked without a product that could wrap
bool too_large(int64_t a, int64_t b) { return b >= kMaxElems || (b > 0 && a > (kMaxElems - 1) / b); }

// The runtime's per-thread last-error slot may hold an earlier, unrelated
// error: it is cleared right before the launches, so that launch_status
// reports only their own failures.
void clear_stale_error() { (void)hipGetLastError(); }

int launch_status() { return hipGetLastError() == hipSuccess ? UE5M3FP4_OK : UE5M3FP4_EHIP; }

}  // namespace

extern "C" {

int ue5m3fp4_quantize_grouped(const uint16_t* x, int64_t x_rows, int64_t cols, int64_t ld, const int32_t* index,
                              int64_t rows, const int32_t* offsets, int64_t experts, const float* tensor_scale,
                              int rounding, uint64_t seed, uint32_t offset, uint8_t* row_codes, uint8_t* row_scales,
                              uint8_t* col_codes, uint8_t* col_scales, float* amax_inout, void* stream) {
    if (x_rows < 0 || cols < 0 || ld < 0 || rows < 0 || experts < 0 || !is01(rounding)) return UE5M3FP4_EINVAL;
    if ((row_codes == nullptr) != (row_scales == nullptr) || (col_codes == nullptr) != (col_scales == nullptr))
        return UE5M3FP4_EINVAL;
    if (rows >= kMaxDim || x_rows >= kMaxDim || cols >= kMaxDim || experts > kMaxExperts) return UE5M3FP4_ERANGE;
    const int64_t padded = rows_padded(rows, experts);
    if (padded >= kMaxDim || too_large(x_rows, ld) || too_large(cols, padded)) return UE5M3FP4_ERANGE;
    if (cols % 16 != 0 || (!index && x_rows != rows)) return UE5M3FP4_ESHAPE;
    if (rows == 0 || cols == 0 || experts == 0) return UE5M3FP4_OK;  // no row to quantize
    const bool outputs = row_codes || col_codes;
    if ((!x && x_rows > 0) || !offsets || (!outputs && !amax_inout) || (outputs && !tensor_scale)) return UE5M3FP4_EINVAL;
    if (row_codes == col_codes && row_codes) return UE5M3FP4_EINVAL;  // one buffer for both
    if (row_scales == col_scales && row_scales) return UE5M3FP4_EINVAL;
    if (ld < cols) return UE5M3FP4_ESHAPE;
    if (ld % 8 != 0) return UE5M3FP4_EALIGN;
    if (!aligned16(x) || !aligned16(row_codes) || !aligned16(row_scales) || !aligned16(col_codes) ||
        !aligned16(col_scales) || !aligned4(index) || !aligned4(offsets) || !aligned4(tensor_scale) ||
        !aligned4(amax_inout))
        return UE5M3FP4_EALIGN;
    const QuantizeGroupedArgs a{x,         x_rows,     cols,      ld,         index,
                                rows,      offsets,    (int)experts, tensor_scale, rounding == UE5M3FP4_SR,
                                seed,      offset,     row_codes, row_scales, col_codes,
                                col_scales, amax_inout};
    clear_stale_error();
    launch_quantize_grouped(a, (hipStream_t)stream);
    return launch_status();
}

int ue5m3fp4_gemm_grouped_nt(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_ts,
                             const uint8_t* b_codes, const uint8_t* b_scales, const float* b_ts, int64_t b_ts_count,
                             const int32_t* offsets, int64_t experts, int64_t rows, int64_t N, int64_t K, void* c,
                             int c_type, float* amax_inout, void* stream) {
    if (experts < 0 || rows < 0 || N < 0 || K < 0 || !is01(c_type)) return UE5M3FP4_EINVAL;
    if (b_ts_count != 1 && b_ts_count != experts) return UE5M3FP4_EINVAL;
    if (amax_inout && c_type != UE5M3FP4_OUT_BF16) return UE5M3FP4_EINVAL;
    if (rows >= kMaxDim || N >= kMaxDim || K >= kMaxK || experts > kMaxExperts) return UE5M3FP4_ERANGE;
    if (too_large(rows, N) || too_large(rows, K) || too_large(N, K) || too_large(experts, N * K)) return UE5M3FP4_ERANGE;
    if (K % 16 != 0) return UE5M3FP4_ESHAPE;
    if (experts == 0 || rows == 0 || N == 0) return UE5M3FP4_OK;  // nothing is read or written
    if (!a_ts || !b_ts || !offsets || !c) return UE5M3FP4_EINVAL;
    if (K > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return UE5M3FP4_EINVAL;
    // weights may begin at any expert of a larger operand, its scales so anywhere, unless K is a multiple of 128
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned8(b_codes) || (K % 128 == 0 && !aligned8(b_scales)) ||
        !aligned16(c) || !aligned4(a_ts) || !aligned4(b_ts) || !aligned4(offsets) || !aligned4(amax_inout))
        return UE5M3FP4_EALIGN;
    const GemmGroupedArgs g{a_codes, a_scales, a_ts, b_codes,      b_scales, b_ts,
                            b_ts_count == 1 ? 0 : 1, offsets, (int)experts, rows,     0, N,
                            K,       c,        c_type == UE5M3FP4_OUT_BF16, amax_inout, 0};
    clear_stale_error();
    launch_gemm_grouped_nt(g, (hipStream_t)stream);
    return launch_status();
}

int ue5m3fp4_gemm_grouped_wgrad(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_ts,
                                const uint8_t* b_codes, const uint8_t* b_scales, const float* b_ts,
                                const int32_t* offsets, int64_t experts, int64_t rows, int64_t M, int64_t N, void* c,
                                int c_type, void* stream) {
    if (experts < 0 || rows < 0 || M < 0 || N < 0 || !is01(c_type)) return UE5M3FP4_EINVAL;
    if (rows >= kMaxDim || M >= kMaxDim || N >= kMaxDim || experts > kMaxExperts) return UE5M3FP4_ERANGE;
    const int64_t padded = rows_padded(rows, experts);
    if (padded >= kMaxK || too_large(M, padded) || too_large(N, padded) || too_large(M, N) || too_large(experts, M * N))
        return UE5M3FP4_ERANGE;
    if (experts == 0 || M == 0 || N == 0) return UE5M3FP4_OK;
    if (!a_ts || !b_ts || !offsets || !c) return UE5M3FP4_EINVAL;
    if (rows > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)) return UE5M3FP4_EINVAL;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) || !aligned16(c) ||
        !aligned4(a_ts) || !aligned4(b_ts) || !aligned4(offsets))
        return UE5M3FP4_EALIGN;
    const GemmGroupedArgs g{a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, 0,       offsets, (int)experts,
                            rows,    M,        N,    0,       c,        c_type == UE5M3FP4_OUT_BF16, nullptr, 0};
    clear_stale_error();
    launch_gemm_grouped_wgrad(g, (hipStream_t)stream);
    return launch_status();
}

int ue5m3fp4_gemm_weight_only(const uint16_t* x, int64_t ldx, const uint8_t* w_codes, const uint8_t* w_scales,
                              const float* w_ts, int64_t w_ts_count, const int32_t* offsets, int64_t experts,
                              int64_t rows, int64_t N, int64_t K, void* out, int out_type, int64_t ldo, void* stream) {
    if (experts < 0 || rows < 0 || N < 0 || K < 0 || ldx < 0 || ldo < 0 || !is01(out_type)) return UE5M3FP4_EINVAL;
    if (!offsets && experts > 1) return UE5M3FP4_EINVAL;
    if (w_ts_count != 1 && w_ts_count != experts) return UE5M3FP4_EINVAL;
    if (rows >= kMaxDim || N >= kMaxDim || K >= kMaxK || experts > kMaxExperts) return UE5M3FP4_ERANGE;
    if (rows <= 1) ldo = N;  // a single row has no stride
    if (rows <= 1 || K == 0) ldx = (K + 7) / 8 * 8;
    if (ldx >= kMaxK || too_large(rows, ldx) || too_large(rows, ldo) || too_large(N, K) || too_large(experts, N * K)) return UE5M3FP4_ERANGE;
    if (K % 16 != 0) return UE5M3FP4_ESHAPE;
    if (experts == 0 || rows == 0 || N == 0) return UE5M3FP4_OK;  // nothing is read or written
    if (!w_ts || !out) return UE5M3FP4_EINVAL;
    if (K > 0 && (!x || !w_codes || !w_scales)) return UE5M3FP4_EINVAL;
    if (ldx < K || ldo < N) return UE5M3FP4_ESHAPE;
    if (ldx % 8 != 0) return UE5M3FP4_EALIGN;
    if (!aligned16(x) || !aligned8(w_codes) || !aligned16(out) || !aligned4(w_ts) || !aligned4(offsets))
        return UE5M3FP4_EALIGN;
    const WeightOnlyArgs a{x,    ldx, w_codes, w_scales, w_ts, w_ts_count == 1 ? 0 : 1, offsets, (int)experts,
                           rows, N,   K,       out,      out_type == UE5M3FP4_OUT_BF16, ldo};
    clear_stale_error();
    launch_gemm_weight_only(a, (hipStream_t)stream);
    return launch_status();
}

}  // extern "C"
