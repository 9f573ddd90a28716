/*
 * mxfp4_fewtoken.h -- C ABI of libmxfp4.so's few-token operators: products
 * of a few BF16 activation rows with MXFP4 weights, and the router and
 * experts of a mixture-of-experts (MoE) layer, on AMD Instinct gfx950
 * (MI355X). They are what a decode step runs where its rows are too few for
 * the 32-row blocks of mxfp4_gemm: the activations stay BF16 (nothing is
 * quantized per call), the weights are MXFP4 in the layout mxfp4_quantize
 * writes (mxfp4.h: codes [rows, K/2], scales [rows, K/32]).
 *
 * Ownership, threading, validation and return codes are those of mxfp4.h:
 * device pointers owned by the caller, nothing allocated, copied or
 * synchronized, work enqueued on `stream` only (so every call can be
 * captured into a HIP graph), every argument checked before anything is
 * enqueued. Buffers that a call writes must not overlap its other buffers.
 *
 * Weights: dq(code, scale) = E2M1(code) * 2^(scale - 127) is taken in BF16,
 * exactly, for scale bytes up to 252, the largest mxfp4_quantize writes
 * (6 * 2^125 is BF16's last binade). Bytes 253 and 254 give infinity where
 * the value passes BF16's range and 255 gives NaN. Results: sums of exact
 * products in FP32, in a fixed order (equal arguments give equal bits).
 * Infinities and NaN in x reach only the outputs of their own row.
 */
#ifndef MXFP4_FEWTOKEN_H
#define MXFP4_FEWTOKEN_H

#include <stdint.h>

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* y[m, n] = sum_k x[m, k] * dq(W[n, k]) for a few rows m.
 * x_bf16 [M, K] BF16, row m at x + m * ldx elements: 16-byte aligned,
 *   ldx >= K and ldx % 8 == 0 (ldx is not read when M == 1)
 * W_codes [N, K/2] 16-byte aligned; W_scales [N, K/32] byte-addressed
 * y [M, N] row-major, BF16 (round to nearest even) or FP32: 4-byte aligned
 * Requires 1 <= M <= 1048560, 1 <= N <= 2^31 - 1, K >= 32, K % 32 == 0,
 * K <= 2^24, each buffer < 2^40 bytes; any M and N, odd ones included. W is
 * read once per 16 rows of x: with many rows quantize them and run
 * mxfp4_gemm. */
int mxfp4_gemv(const void* x_bf16, int64_t ldx, const void* W_codes, const void* W_scales,
               int64_t M, int64_t N, int64_t K, int out_dtype, void* y, void* stream);

/* Router of an MoE layer: for each of T tokens
 *   l[e] = sum_h x[h] * R[e, h]  (64-bit sums),  p = softmax(l) over E
 *   ids[j]     = the expert with the (j + 1)-th largest l, j < top_k; of
 *                equal ones the lowest index first
 *   weights[j] = p[ids[j]], divided by the sum of the top_k chosen ones when
 *                renormalize is 1; in 64 bits, rounded to FP32 once
 * x_bf16 [T, H] as mxfp4_gemv's x; router_bf16 [E, H] BF16, 16-byte aligned
 * ids [T, top_k] int32, weights [T, top_k] FP32: 4-byte aligned
 * workspace: mxfp4_moe_route_workspace bytes, 16-byte aligned, any content;
 *   not to be used by another call until this one has run. It is 0 bytes,
 *   and workspace may be NULL, where the sizes need none
 * Requires 1 <= T <= 65535, H % 8 == 0, 8 <= H <= 2^24, 1 <= E <= 1024,
 * 1 <= top_k <= min(E, 32), renormalize 0 or 1. A token with NaN logits gets
 * distinct ids below E (NaN sorts last) and NaN weights. */
int mxfp4_moe_route_workspace(int64_t T, int64_t H, int64_t E, int64_t* bytes);
int mxfp4_moe_route(const void* x_bf16, int64_t ldx, const void* router_bf16, int64_t T,
                    int64_t H, int64_t E, int64_t top_k, int renormalize, void* ids,
                    void* weights, void* workspace, void* stream);

/* The experts of an MoE layer for T routed tokens:
 *   y[t] = sum_j weights[t, j] * W2_e (silu(Wg_e x[t]) * (Wu_e x[t])),
 *   e = ids[t, j], silu(z) = z / (1 + exp(-z)), in FP32 up to y, whatever
 *   its type and however many tokens there are (several tokens' activations
 *   may lose bits below 2^-133).
 * An id outside 0 .. E - 1 adds nothing and its weight is not read into the
 * sum (an expert that another device holds); a token with no expert here
 * gets zeros. A token may name an expert more than once.
 * x_bf16 [T, H] as mxfp4_gemv's x
 * ids [T, top_k] int32, weights [T, top_k] FP32: 4-byte aligned
 * W13 codes [E, 2 I, H/2], scales [E, 2 I, H/32]: per expert the stacked
 *   [W_gate; W_up], I rows each (the order of mxfp4_gemm_swiglu)
 * W2 codes [E, H, I/2], scales [E, H, I/32]; codes 16-byte aligned, scales
 *   byte-addressed
 * y [T, H] BF16 or FP32: 4-byte aligned
 * workspace: mxfp4_moe_workspace bytes, 16-byte aligned, any content; not to
 *   be used by another call until this one has run
 * Requires T >= 1, 1 <= top_k <= 32, T * top_k <= 1024, H and I >= 32 and
 * % 32 == 0, H and I <= 2^20, 1 <= E <= 1024, each buffer < 2^40 bytes. */
int mxfp4_moe_workspace(int64_t T, int64_t H, int64_t I, int64_t top_k, int64_t* bytes);
int mxfp4_moe(const void* x_bf16, int64_t ldx, const void* ids, const void* weights,
              const void* W13_codes, const void* W13_scales, const void* W2_codes,
              const void* W2_scales, int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k,
              int out_dtype, void* y, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_FEWTOKEN_H */
