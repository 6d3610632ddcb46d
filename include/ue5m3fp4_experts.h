/*
 * libue5m3fp4_experts -- the FP4 linears of routed experts, and products of
 * unquantized tokens with FP4 weights, for AMD Instinct MI355X (gfx950):
 *
 *   - quantization of rows that are grouped by expert (ragged sizes), with an
 *     optional gather of the rows from the tokens they were routed from;
 *   - the three training GEMMs of the experts' linears on such operands;
 *   - bf16 tokens times FP4 weights, of one linear or of routed experts, for
 *     the few tokens of a generation step.
 * Formats, arithmetic and operand layouts are those of include/ue5m3fp4.h
 * ("UE5M3 FP4 Block Scaling for Stable Language Model Pretraining", arXiv
 * 2609.02846, abstract: FP4 in all eligible internal linears, of which an
 * expert's are some).
 *
 * Groups.  The rows of a matrix of `rows` rows are sorted by expert;
 * offsets, int32 [experts + 1] on the device, says which: expert g owns the
 * rows offsets[g] .. offsets[g + 1] - 1 (none where they are equal).  Rows
 * before offsets[0] and from offsets[experts] on belong to no expert: they are
 * not read, and outputs keep what they held there.  The values are not known
 * on the host and are not checked there; kernels take offsets[g] as clamped to
 * [0, rows] and offsets[g + 1] to [offsets[g], rows], so no value makes them
 * access memory outside the operands, but offsets that decrease leave the
 * contents of the outputs undefined.
 *
 * Grouped transposed operands.  Blocks of 16 rows must not span two experts,
 * and GEMM steps are 128 deep, so expert g's rows stand in a transposed
 * operand (cols x rows_padded) from column
 *     p_g = 128 * (ceil(offsets[g] / 128) + g)
 * on, followed by quantized zeros (codes and scales 0 under any tensor scale
 * but 0 and NaN) up to the next multiple of 128 columns; rows_padded = 128 *
 * (ceil(rows / 128) + experts).  Columns of no expert are neither written nor
 * read.  In other words: inside these column ranges the operand is the
 * transposed output of ue5m3fp4_quantize_blockscale for the rows_padded x cols
 * matrix that holds the experts' rows at their p_g and zeros elsewhere
 * (stochastic rounding draws for that matrix too).
 *
 * Expert weights.  codes [experts][R][C / 2], scales [experts][R][C / 16],
 * and one tensor scale for all experts or one for each.  They may be some
 * experts of a larger operand: codes have to be 8-byte aligned, scales 8-byte
 * where C is a multiple of 128, else not at all.
 *
 * Sums.  Products are exact and sums are fp32.  A sum passes at most 2048
 * roundings one after another: longer contractions are joined from shorter
 * sums whose roundings are carried on.  So a result is off by at most 2^-13 of
 * |ts| sum|a b| however long the contraction and whatever the terms, and by
 * less than 1e-5 of it where they are not alike (rounding to bf16 comes on top).
 *
 * Conventions: those of include/ue5m3fp4.h -- device pointers owned by the
 * caller, every argument checked on the host before any HIP call, work
 * enqueued on `stream` of the current device, nothing allocated, synchronized
 * or kept; other array base pointers 16-byte aligned, scalars, offsets and
 * indices 4-byte aligned; sizes of 0 are valid and launch nothing (except GEMMs with
 * an empty contraction, which write zeros).  At most 65536 experts (ERANGE).
 */
#ifndef UE5M3FP4_EXPERTS_H
#define UE5M3FP4_EXPERTS_H

#include "ue5m3fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of an output. */
enum ue5m3fp4_output_type { UE5M3FP4_OUT_BF16 = 0, UE5M3FP4_OUT_F32 = 1 };

/* Quantize rows grouped by expert under the fp32 tensor scale *tensor_scale.
 *   x: bf16, x_rows x cols, row stride ld elements;
 *   index: nullable device int32 [rows]: row i of the grouped matrix is
 *       x[index[i]] (a token that several experts take is read for each; an
 *       index outside [0, x_rows) gives a row of zeros).  Without it the
 *       grouped matrix is x itself and x_rows must equal rows (ESHAPE);
 *   row_codes / row_scales: the row-wise operand, [rows][cols / 2] and
 *       [rows][cols / 16], as ue5m3fp4_quantize_blockscale writes it;
 *   col_codes / col_scales: the grouped transposed operand, [cols]
 *       [rows_padded / 2] and [cols][rows_padded / 16];
 *   rounding, seed, offset: as ue5m3fp4_quantize_blockscale (the row-wise
 *       stream counts elements of the rows x cols matrix, the transposed one
 *       those of the cols x rows_padded matrix);
 *   amax_inout: nullable; receives max(*amax_inout, max|x|) over the experts'
 *       rows (a NaN propagates).  It starts at 0 or an earlier amax: values with
 *       a sign, -0 included, are kept as they are (so in the products, too).
 * Each pair is both NULL or both non-NULL, at least one of the pairs and
 * amax_inout non-NULL; tensor_scale may be NULL without pairs.
 * cols % 16 == 0 (ESHAPE), ld >= cols (ESHAPE), ld % 8 == 0 (EALIGN); rows,
 * x_rows, cols, rows_padded < 2^31, x_rows * ld and cols * rows_padded < 2^40
 * (ERANGE).  Inputs and outputs must not overlap. */
UE5M3FP4_API int ue5m3fp4_quantize_grouped(const uint16_t* x, int64_t x_rows, int64_t cols, int64_t ld,
                                           const int32_t* index, int64_t rows, const int32_t* offsets,
                                           int64_t experts, const float* tensor_scale, int rounding, uint64_t seed,
                                           uint32_t offset, uint8_t* row_codes, uint8_t* row_scales,
                                           uint8_t* col_codes, uint8_t* col_scales, float* amax_inout, void* stream);

/* fprop and dgrad of the experts' linears: for the rows i of expert g
 *   C[i][j] = (tsA * tsB_g) * sum_k A(i, k) * B_g(j, k),  fp32 accumulation,
 * as ue5m3fp4_gemm_nt does for one matrix.
 *   a: rows x K, row-wise (X, or dY);
 *   b: expert weights [experts][N][K] (W row-wise, or W's transposed output);
 *   b_ts: b_ts_count device fp32 values, 1 or `experts` of them (EINVAL);
 *   c: [rows][N], bf16 (rounded to nearest even) or fp32;
 *   amax_inout: nullable, for bf16 outputs only (EINVAL): receives
 *       max(*amax_inout, max|C|) over the values stored (a NaN propagates).
 * K % 16 == 0 (ESHAPE); rows, N < 2^31, K < 2^24, rows * N, rows * K and
 * experts * N * K < 2^40 (ERANGE).  c must not overlap the operands. */
UE5M3FP4_API int ue5m3fp4_gemm_grouped_nt(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_ts,
                                          const uint8_t* b_codes, const uint8_t* b_scales, const float* b_ts,
                                          int64_t b_ts_count, const int32_t* offsets, int64_t experts, int64_t rows,
                                          int64_t N, int64_t K, void* c, int c_type, float* amax_inout, void* stream);

/* wgrad of the experts' linears: for every expert g, over the columns p that
 * its rows have in the grouped transposed operands,
 *   C_g[i][j] = (tsA * tsB) * sum_p A(i, p) * B(j, p),  fp32 accumulation.
 *   a: M x rows_padded (dY's transposed output); b: N x rows_padded (X's);
 *   rows: those that the operands were quantized from (offsets are clamped to
 *       them in both places, so the numbers have to agree);
 *   c: [experts][M][N], bf16 or fp32; an expert without rows gets zeros.
 * M, N < 2^31, rows_padded < 2^24; M * rows_padded, N * rows_padded and experts
 * * M * N < 2^40 (ERANGE). */
UE5M3FP4_API int ue5m3fp4_gemm_grouped_wgrad(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_ts,
                                             const uint8_t* b_codes, const uint8_t* b_scales, const float* b_ts,
                                             const int32_t* offsets, int64_t experts, int64_t rows, int64_t M,
                                             int64_t N, void* c, int c_type, void* stream);

/* Tokens that stay in bf16 times FP4 weights:
 *   out[i][j] = ts_g * sum_k x[i][k] * W_g(j, k),
 * products exact (fp32 sums), rounded once to out's type; made for the few
 * rows (1 to about 64 per expert) of a generation step, any number is valid.
 *   x: bf16, rows x K, row stride ldx elements (ldx >= K: ESHAPE; ldx % 8 ==
 *       0: EALIGN; both only where rows > 1).  Subnormal elements may count
 *       as 0;
 *   w: one matrix N x K row-wise (offsets NULL, experts 1), or expert weights
 *       [experts][N][K] with the rows grouped by offsets;
 *   w_ts: w_ts_count device fp32 values, 1 or `experts` of them (EINVAL);
 *   out: [rows][N], row stride ldo elements (ldo >= N where rows > 1: ESHAPE).
 * K % 16 == 0 (ESHAPE); rows, N < 2^31, K, ldx < 2^24, rows * ldx, rows * ldo
 * and experts * N * K < 2^40 (ERANGE).  out must not overlap the inputs. */
UE5M3FP4_API int ue5m3fp4_gemm_weight_only(const uint16_t* x, int64_t ldx, const uint8_t* w_codes,
                                           const uint8_t* w_scales, const float* w_ts, int64_t w_ts_count,
                                           const int32_t* offsets, int64_t experts, int64_t rows, int64_t N, int64_t K,
                                           void* out, int out_type, int64_t ldo, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* UE5M3FP4_EXPERTS_H */
