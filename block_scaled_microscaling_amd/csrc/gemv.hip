// y = x dq(W)^T for a few BF16 rows x and an MXFP4 weight W [N, K].
//
// Mathematics: y[m, n] = sum_k x[m, k] E2M1(code[n, k]) 2^(scale[n, k/32] -
// 127). A weight value has two significand bits, so it is exact in BF16 and
// every product is exact in FP32; only the FP32 sums round.
//
// What bounds it: the weight's 17/32 byte per element is read once, for 2 M
// flop per element: HBM for every M here.
//
// Work split: a workgroup of 8 waves owns 16 weight rows and 16 tokens; the
// K chunks go round the waves and the 8 partial tiles are summed in LDS in
// wave order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

template <bool kOutFp32>
__global__ __launch_bounds__(kThreads) void gemv_kernel(const uint8_t* __restrict__ x, int64_t ldx,
                                                        const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, int M,
                                                        int N, int KB, void* __restrict__ y) {
  __shared__ __align__(16) float red[kWaves * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n0 = blockIdx.x * kFewTile;
  const int m0 = blockIdx.y * kFewTile;
  // Rows and tokens past the end re-read the last one; they are not stored.
  const int n = min(n0 + (lane & 15), N - 1);
  const int m = min(m0 + (lane & 15), M - 1);
  const uint8_t* wc[1] = {codes + (int64_t)n * KB * 16};
  const uint8_t* ws[1] = {scales + (int64_t)n * KB};
  v4f_t acc[1] = {v4f_t{}};
  few_mac<1>(wc, ws, x + (int64_t)m * ldx * 2, KB, wave, kWaves, lane >> 4, acc);
  // Output (row 4 g + v, token t) at 64 v + 16 g + t of the wave's part.
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave * 256 + v * 64 + lane] = acc[0][v];
  __syncthreads();
  if (threadIdx.x < 256) {
    // Thread i: row i % 16 of token i / 16, so a token's rows store together.
    const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
    const int at = (r & 3) * 64 + (r >> 2) * 16 + t;
    float sum = red[at];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w * 256 + at];
    if (n0 + r < N && m0 + t < M) {
      const int64_t o = (int64_t)(m0 + t) * N + n0 + r;
      if constexpr (kOutFp32)
        static_cast<float*>(y)[o] = sum;
      else
        static_cast<uint16_t*>(y)[o] = (uint16_t)pack_bf16x2(sum, sum);
    }
  }
}

}  // namespace

hipError_t launch_gemv(const void* x, int64_t ldx, const void* codes, const void* scales, int M,
                       int N, int K, bool out_fp32, void* y, hipStream_t stream) {
  const dim3 grid((uint32_t)(((int64_t)N + kFewTile - 1) / kFewTile), (M + kFewTile - 1) / kFewTile);
  const auto* xb = static_cast<const uint8_t*>(x);
  const auto* wc = static_cast<const uint8_t*>(codes);
  const auto* ws = static_cast<const uint8_t*>(scales);
  if (out_fp32)
    hipLaunchKernelGGL((gemv_kernel<true>), grid, dim3(kThreads), 0, stream, xb, ldx, wc, ws, M, N,
                       K / 32, y);
  else
    hipLaunchKernelGGL((gemv_kernel<false>), grid, dim3(kThreads), 0, stream, xb, ldx, wc, ws, M,
                       N, K / 32, y);
  return hipGetLastError();
}

}  // namespace mxfp4
