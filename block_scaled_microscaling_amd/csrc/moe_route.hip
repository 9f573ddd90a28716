// Router of a mixture-of-experts layer: logits, softmax and top k.
//
// Mathematics: l[t, e] = sum_h x[t, h] R[e, h] in 64 bits (products of BF16
// pairs are exact; which of two close experts wins hangs on a logit's last
// bits, and 64-bit sums make that independent of the summation order for
// all practical inputs), p = exp(l - max l) / sum exp(l - max l) in FP32.
//
// Two kernels: the first writes the logits (one wave per token and expert),
// the second takes one wave per token.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxPerLane = 16;  // 1024 experts over 64 lanes

__device__ __forceinline__ double lo_bf16(uint32_t w) { return (double)__uint_as_float(w << 16); }
__device__ __forceinline__ double hi_bf16(uint32_t w) {
  return (double)__uint_as_float(w & 0xFFFF0000u);
}

__global__ __launch_bounds__(kThreads) void route_logits_kernel(const uint8_t* __restrict__ x,
                                                                int64_t ldx,
                                                                const uint8_t* __restrict__ router,
                                                                int T, int H, int E,
                                                                double* __restrict__ logits) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int e = blockIdx.x;
  const int t = blockIdx.y * kWaves + wave;
  if (t >= T) return;
  const auto* xr = reinterpret_cast<const u32x4_t*>(x + (int64_t)t * ldx * 2);
  const auto* rr = reinterpret_cast<const u32x4_t*>(router + (int64_t)e * H * 2);
  double sum = 0.0;
  for (int i = lane; i < H / 8; i += 64) {
    const u32x4_t a = xr[i], b = rr[i];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t aw = a[q], bw = b[q];
      sum = fma(lo_bf16(aw), lo_bf16(bw), sum);
      sum = fma(hi_bf16(aw), hi_bf16(bw), sum);
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) logits[(int64_t)t * E + e] = sum;
}

// A logit as an integer that orders as it does: NaN below everything else,
// and INT64_MIN is left free for an expert already taken.
__device__ __forceinline__ int64_t order_key(double v) {
  if (v != v) return INT64_MIN + 1;
  const int64_t b = __double_as_longlong(v + 0.0);  // -0 counts as +0
  return b >= 0 ? b : (b ^ INT64_MAX);
}

__global__ __launch_bounds__(64) void route_top_kernel(const double* __restrict__ logits, int E,
                                                       int top_k, int renormalize,
                                                       int32_t* __restrict__ ids,
                                                       float* __restrict__ weights) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const double* l = logits + t * E;
  int64_t key[kMaxPerLane];
  double top = 0.0;
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    const int e = i * 64 + lane;
    key[i] = e < E ? order_key(l[e]) : INT64_MIN;
  }
  float chosen = 0.0f, mine = 0.0f;
  int mine_id = 0;
  for (int j = 0; j < top_k; ++j) {
    int64_t best = INT64_MIN;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * 64 + lane;
      }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const int64_t ob = __shfl_xor((long long)best, d);
      const int oa = __shfl_xor(at, d);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (j == 0) {
      // The largest logit is known: the softmax's sum.
      top = l[at];
#pragma unroll
      for (int i = 0; i < kMaxPerLane; ++i)
        if (i * 64 + lane < E) total += expf((float)(l[i * 64 + lane] - top));
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) total += __shfl_xor(total, d);
    }
    const float p = expf((float)(l[at] - top)) / total;
    chosen += p;
    if (lane == j) {
      mine = p;
      mine_id = at;
    }
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i)
      if (at == i * 64 + lane) key[i] = INT64_MIN;
  }
  if (lane < top_k) {
    ids[t * top_k + lane] = mine_id;
    weights[t * top_k + lane] = renormalize ? mine / chosen : mine;
  }
}

}  // namespace

hipError_t launch_moe_route(const void* x, int64_t ldx, const void* router, int T, int H, int E,
                            int top_k, bool renormalize, int32_t* ids, float* weights,
                            double* logits, hipStream_t stream) {
  hipLaunchKernelGGL(route_logits_kernel, dim3(E, (T + kWaves - 1) / kWaves), dim3(kThreads), 0,
                     stream, static_cast<const uint8_t*>(x), ldx,
                     static_cast<const uint8_t*>(router), T, H, E, logits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(route_top_kernel, dim3(T), dim3(64), 0, stream, logits, E, top_k,
                     renormalize ? 1 : 0, ids, weights);
  return hipGetLastError();
}

}  // namespace mxfp4
