/*
 * mxfp4_fp8.h -- C ABI of libmxfp4.so's FP8 operators on AMD Instinct gfx950
 * (MI355X): quantize, GEMM and the gated MLP's forward and backward passes on
 * 8-bit floating point with one scale for each block of 128, beside the MXFP4
 * ones of mxfp4.h. They serve the layers and gradients that do not stand
 * 4 bits, and weights that are stored this way.
 *
 * Format. Codes are OCP E4M3 (largest 448) or E5M2 (largest 57344), one byte
 * each, row-major. A scale covers 128 consecutive elements of a row ("rows",
 * scales [rows, ceil(K / 128)]) or a 128 x 128 block ("blocks", scales
 * [ceil(rows / 128), ceil(K / 128)]); the last block of a row or column may be
 * short. Scales are UE8M0 bytes, 2^(byte - 127), 255 = NaN, or FP32.
 *
 * Ownership, threading, validation and return codes are those of mxfp4.h:
 * device pointers owned by the caller, nothing allocated, copied or
 * synchronized, work enqueued on `stream` only (so every call can be captured
 * into a HIP graph), every argument checked before anything is enqueued.
 * Buffers that a call writes must not overlap its other buffers. Equal
 * arguments give equal bits. In every entry point sizes are at least 1 and at
 * most 2^31 - 256, K (and H, I) at most 2^24 and a multiple of 16, each buffer
 * is below 2^40 bytes; codes, BF16 and FP32 matrices are 16-byte aligned,
 * UE8M0 scales byte-addressed, FP32 scales 4-byte aligned.
 */
#ifndef MXFP4_FP8_H
#define MXFP4_FP8_H

#include <stdint.h>

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum mxfp4_fp8_type { MXFP4_FP8_E4M3 = 0, MXFP4_FP8_E5M2 = 1 };
enum mxfp4_fp8_scale { MXFP4_SCALE_UE8M0 = 0, MXFP4_SCALE_FP32 = 1 };

/* BF16 -> FP8, block_rows = 1 (rows) or 128 (blocks). For each block:
 *   amax  = max |x| over its finite values
 *   e     = the smallest integer with amax <= T 2^e, T = 448 or 57344,
 *           clamped to [-126, 127] (-126 where amax is 0)
 *   scale = 2^e, as UE8M0 byte e + 127 or as FP32
 *   code  = x / 2^e rounded to nearest even
 * NaN gives NaN; an infinity gives NaN (E4M3) or infinity (E5M2).
 * x_bf16 [M, K], row m at x + m * ldx elements: ldx >= K, ldx % 8 == 0 (not
 *   read when M == 1)
 * codes [M, K], scales [M, ceil(K/128)] or [ceil(M/128), ceil(K/128)] */
int mxfp4_quantize_fp8(const void* x_bf16, int64_t ldx, int64_t M, int64_t K, int64_t block_rows,
                       int code_type, int scale_type, void* codes, void* scales, void* stream);

/* The same of x and of its transpose in one pass. With Mp = M rounded up to a
 * multiple of 16:
 * codes_t [K, Mp], zeros in columns M .. Mp - 1; scales_t [K, ceil(M/128)], or
 * with block_rows 128 the transpose of scales, [ceil(K/128), ceil(M/128)].
 * Requires M <= 2^24. */
int mxfp4_quantize_fp8_2d(const void* x_bf16, int64_t ldx, int64_t M, int64_t K,
                          int64_t block_rows, int code_type, int scale_type, void* codes,
                          void* scales, void* codes_t, void* scales_t, void* stream);

/* C[m, n] = sum_k dq(A[m, k]) dq(B[n, k]), FP32 sums. FP32 results add exact
 * products. BF16 results of large products use the FP8 matrix instructions,
 * which cut eight neighbouring products off 2^-14 below the largest of them:
 * each eight may be off by 2^-10 of their max |a| max |b|, a typical sum by
 * 1.3e-5 of itself, before the rounding to BF16.
 * A_codes [M, K] of A_type, A_scales [M, ceil(K/128)]
 * B_codes [N, K] E4M3, B_scales [ceil(N/128), ceil(K/128)] (B_block_rows 128)
 *   or [N, ceil(K/128)] (B_block_rows 1, with UE8M0 scales only)
 * scale_type: of both operands
 * C [M, N], BF16 (round to nearest even) or FP32; any M and N. */
int mxfp4_gemm_fp8(const void* A_codes, int A_type, const void* A_scales, const void* B_codes,
                   const void* B_scales, int scale_type, int64_t B_block_rows, int64_t M,
                   int64_t N, int64_t K, int out_dtype, void* C, void* stream);

/* The gate+up product of a gated MLP with its activation, for A = the layer's
 * input [M, K] and the stacked W13 = [W_gate; W_up] [2 I, K], both E4M3 with
 * UE8M0 scales, W13's in blocks; I % 128 == 0:
 *   g = A W_gate^T, u = A W_up^T, act = silu(g) u in FP32, rounded to BF16,
 *   then quantized as mxfp4_quantize_fp8 does (rows, E4M3, UE8M0)
 * codes [M, I], scales [M, I/128]: the down product's A operand
 * act_bf16 [M, I]: the BF16 act, or NULL
 * gu_bf16 [M, 2 I]: g and u rounded to BF16, which the backward pass takes,
 *   or NULL
 * workspace: mxfp4_gemm_fp8_swiglu_workspace bytes, 16-byte aligned, any
 *   content; not to be used by another call until this one has run. It is 0
 *   bytes, and workspace may be NULL, where the sizes need none. */
int mxfp4_gemm_fp8_swiglu_workspace(int64_t M, int64_t I, int64_t K, int64_t* bytes);
int mxfp4_gemm_fp8_swiglu(const void* A_codes, const void* A_scales, const void* W13_codes,
                          const void* W13_scales, int64_t M, int64_t I, int64_t K, void* codes,
                          void* scales, void* act_bf16, void* gu_bf16, void* workspace,
                          void* stream);

/* The backward pass of act = silu(g) u, quantized for the two products that
 * follow it. With s = 1 / (1 + exp(-g)), in FP32:
 *   dg = dact u s (1 + g (1 - s)),   du = dact g s,   dgu = [dg, du]
 * dact_bf16 [M, I], gu_bf16 [M, 2 I]; I % 128 == 0, M <= 2^24
 * codes [M, 2 I], scales [M, 2 I/128]: dgu quantized from FP32 as above (rows,
 *   UE8M0), the A operand of dx = dgu W13
 * codes_t [2 I, Mp], scales_t [2 I, ceil(M/128)]: the same of dgu^T with zeros
 *   in columns M .. Mp - 1, Mp = M rounded up to 16, the A operand of
 *   dW13 = dgu^T x */
int mxfp4_swiglu_fp8_backward(const void* dact_bf16, const void* gu_bf16, int64_t M, int64_t I,
                              int code_type, void* codes, void* scales, void* codes_t,
                              void* scales_t, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_FP8_H */
