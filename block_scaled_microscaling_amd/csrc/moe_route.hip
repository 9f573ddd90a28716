// Router of a mixture-of-experts layer: logits, softmax and top k.
//
// Mathematics: l[t, e] = sum_h x[t, h] R[e, h] in 64 bits (products of BF16
// pairs are exact; which of two close experts wins hangs on a logit's last
// bits, and 64-bit sums make that independent of the summation order for
// all practical inputs), p = exp(l - max l) / sum exp(l - max l) in 64 bits too,
// rounded once: FP32 from the differences on is 2 to 7% faster (1 token x 4096,
// 8 experts 3.65 against 3.80 us, 1 x 512, 256 experts 6.65 against 7.15) but
// off by 2 to 3 times as much, and by 2^-24 of a far logit's distance.
//
// What bounds it: a few tokens' launches and latencies (1 token x 4096, 8
// experts 3.7 us; 64 tokens x 4096, 128 experts 5.0 + 4.2), many tokens' 2 T E
// H flop of 64-bit arithmetic (512 tokens x 4096, 128 experts 21 us). The
// bytes are few.
//
// Few experts: one workgroup a token does it all (one launch). Otherwise the
// logits are tiles of v_mfma_f64_16x16x4_f64 whose K is split over
// workgroups, and the second kernel, one wave a token, adds the splits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

typedef double v4d_t __attribute__((ext_vector_type(4)));

constexpr int kOneWaves = 16;        // of the one-launch kernel
constexpr int kOneMaxExperts = 128;  // 8 a wave
constexpr int kTile = 16;            // tokens and experts of an MFMA
constexpr int kTileWaves = 8;
constexpr int kMaxSplits = 8;

__device__ __forceinline__ double lo_bf16(uint32_t w) { return (double)__uint_as_float(w << 16); }
__device__ __forceinline__ double hi_bf16(uint32_t w) {
  return (double)__uint_as_float(w & 0xFFFF0000u);
}

// A logit as an integer that orders as it does: NaN below everything else,
// and INT64_MIN is left free for an expert already taken.
__device__ __forceinline__ int64_t order_key(double v) {
  if (v != v) return INT64_MIN + 1;
  const int64_t b = __double_as_longlong(v + 0.0);  // -0 counts as +0
  return b >= 0 ? b : (b ^ INT64_MAX);
}
__device__ __forceinline__ double of_order_key(int64_t k) {
  if (k == INT64_MIN + 1) return __longlong_as_double(0x7FF8000000000000ll);
  return __longlong_as_double(k >= 0 ? k : (k ^ INT64_MAX));
}

// A reduction over the wave, its result in every lane: four DPP steps within
// 16 lanes, then the halves of 32 and of 64.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
}
template <int kCtrl>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  return (uint64_t)dpp32<kCtrl>((uint32_t)(v >> 32)) << 32 | dpp32<kCtrl>((uint32_t)v);
}
template <class Op>
__device__ __forceinline__ uint64_t wave_reduce64(uint64_t v, Op op) {
  v = op(v, dpp64<0xB1>(v));   // quad_perm [1,0,3,2]
  v = op(v, dpp64<0x4E>(v));   // quad_perm [2,3,0,1]
  v = op(v, dpp64<0x141>(v));  // row_half_mirror
  v = op(v, dpp64<0x140>(v));  // row_mirror
  auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  auto hi =
      __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  v = op((uint64_t)hi[0] << 32 | lo[0], (uint64_t)hi[1] << 32 | lo[1]);
  lo = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  hi = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  return op((uint64_t)hi[0] << 32 | lo[0], (uint64_t)hi[1] << 32 | lo[1]);
}
__device__ __forceinline__ double wave_sum(double v) {
  return __longlong_as_double((int64_t)wave_reduce64(
      (uint64_t)__double_as_longlong(v), [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(__longlong_as_double((int64_t)a) +
                                              __longlong_as_double((int64_t)b));
      }));
}
__device__ __forceinline__ int64_t wave_max(int64_t v) {
  return (int64_t)wave_reduce64((uint64_t)v, [](uint64_t a, uint64_t b) {
    return (int64_t)a > (int64_t)b ? a : b;
  });
}

// One wave: softmax and top k of the logits l[i] of experts 64 i + lane
// (those from E on do not count).
template <int kPerLane>
__device__ __forceinline__ void choose(const double (&l)[kPerLane], int E, int top_k,
                                       int renormalize, int32_t* __restrict__ ids,
                                       float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  int64_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) key[i] = i * 64 + lane < E ? order_key(l[i]) : INT64_MIN;
  int64_t mine_key = INT64_MIN, top_key = INT64_MIN;
  int mine_id = 0;
  for (int j = 0; j < top_k; ++j) {
    int64_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max(best);
    // The lowest index that has it.
    int at = 0;
#pragma unroll
    for (int i = kPerLane - 1; i >= 0; --i) {
      const uint64_t m = __ballot(key[i] == best);
      if (m) at = i * 64 + __ffsll((unsigned long long)m) - 1;
    }
    if (j == 0) top_key = best;
    if (lane == j) {
      mine_key = best;
      mine_id = at;
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (at == i * 64 + lane) key[i] = INT64_MIN;
  }
  const double top = of_order_key(top_key);
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)
    if (i * 64 + lane < E) total += exp(l[i] - top);
  total = wave_sum(total);
  const double p = lane < top_k ? exp(of_order_key(mine_key) - top) : 0.0;
  const double sum = renormalize ? wave_sum(p) : total;
  if (lane < top_k) {
    ids[lane] = mine_id;
    weights[lane] = (float)(p / sum);
  }
}

// Lane sums of four experts -> the total of expert r in lanes 16 r .. 16 r + 15.
__device__ __forceinline__ double sum_four(const double (&v)[4]) {
  const auto merge = [](double a, double b, auto swap) {
    const uint64_t x = (uint64_t)__double_as_longlong(a), y = (uint64_t)__double_as_longlong(b);
    const auto lo = swap((uint32_t)x, (uint32_t)y);
    const auto hi = swap((uint32_t)(x >> 32), (uint32_t)(y >> 32));
    return __longlong_as_double((int64_t)((uint64_t)hi[0] << 32 | lo[0])) +
           __longlong_as_double((int64_t)((uint64_t)hi[1] << 32 | lo[1]));
  };
  const auto swap32 = [](uint32_t a, uint32_t b) {
    return __builtin_amdgcn_permlane32_swap(a, b, false, false);
  };
  const auto swap16 = [](uint32_t a, uint32_t b) {
    return __builtin_amdgcn_permlane16_swap(a, b, false, false);
  };
  double s = merge(merge(v[0], v[2], swap32), merge(v[1], v[3], swap32), swap16);
  const auto add = [](double a, uint64_t b) { return a + __longlong_as_double((int64_t)b); };
  s = add(s, dpp64<0xB1>((uint64_t)__double_as_longlong(s)));
  s = add(s, dpp64<0x4E>((uint64_t)__double_as_longlong(s)));
  s = add(s, dpp64<0x141>((uint64_t)__double_as_longlong(s)));
  return add(s, dpp64<0x140>((uint64_t)__double_as_longlong(s)));
}

// One launch: each wave takes 4 kPerLane of the token's experts or, with few
// experts, a part of H for them; wave 0 adds the parts and chooses. So every
// wave's loads go out at once (7 tokens x 296, 120 experts: four experts after
// four 8.2 us a call, all at once 6.3), and four sums are reduced as one (7
// tokens x 920, 7 experts 4.5 -> 3.7 us).
template <int kPerLane>
__global__ __launch_bounds__(64 * kOneWaves) void route_one_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const uint8_t* __restrict__ router, int H, int E,
    int top_k, int renormalize, int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr int kExperts = 4 * kPerLane;
  __shared__ double part[kOneWaves * kExperts];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int groups = (E + kExperts - 1) / kExperts;
  const int parts = kOneWaves / groups;
  const int64_t t = blockIdx.x;
  const auto* xr = reinterpret_cast<const u32x4_t*>(x + t * ldx * 2);
  const int group = wave / parts, p = wave - group * parts;
  if (group < groups) {
    double sum[kPerLane][4] = {};
    for (int i = p * 64 + lane; i < H / 8; i += parts * 64) {
      const u32x4_t a = xr[i];
      u32x4_t b[kPerLane][4];
#pragma unroll
      for (int n = 0; n < kExperts; ++n) {
        const int e = min(group * kExperts + n, E - 1);
        b[n / 4][n % 4] = reinterpret_cast<const u32x4_t*>(router + (int64_t)e * H * 2)[i];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t aw = a[q];
        const double a0 = lo_bf16(aw), a1 = hi_bf16(aw);
#pragma unroll
        for (int n = 0; n < kExperts; ++n) {
          const uint32_t bw = b[n / 4][n % 4][q];
          double& s = sum[n / 4][n % 4];
          s = fma(a0, lo_bf16(bw), s);
          s = fma(a1, hi_bf16(bw), s);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kPerLane; ++n) {
      const double s = sum_four(sum[n]);
      const int e = group * kExperts + 4 * n + (lane >> 4);
      if ((lane & 15) == 0 && e < E) part[p * E + e] = s;
    }
  }
  __syncthreads();
  if (wave != 0) return;
  double l[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = i * 64 + lane;
    l[i] = 0.0;
    if (e < E)
      for (int p = 0; p < parts; ++p) l[i] += part[p * E + e];
  }
  choose(l, E, top_k, renormalize, ids + t * top_k, weights + t * top_k);
}

// Partial logits [split][T][E]: a workgroup takes 16 tokens, 16 experts and
// every gridDim.z-th share of K. Lane l has 8 consecutive h of expert and
// token l % 16, h group l / 16 of 32; element i of the eight feeds the i-th
// MFMA, whose accumulator register v of lane l is (expert 4 v + l / 16, token
// l % 16).
__global__ __launch_bounds__(64 * kTileWaves) void route_logits_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const uint8_t* __restrict__ router, int T, int H,
    int E, double* __restrict__ logits) {
  __shared__ double red[kTileWaves * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int e0 = blockIdx.x * kTile, t0 = blockIdx.y * kTile;
  // Tokens and experts past the end re-read the last one; they are not stored.
  const int64_t t = min(t0 + (lane & 15), T - 1), e = min(e0 + (lane & 15), E - 1);
  const auto* xr = reinterpret_cast<const u32x4_t*>(x + t * ldx * 2);
  const auto* rr = reinterpret_cast<const u32x4_t*>(router + e * H * 2);
  v4d_t acc = {};
  const int stride = kTileWaves * gridDim.z * 4;
#pragma unroll 2
  for (int c = (blockIdx.z * kTileWaves + wave) * 4; c < H / 8; c += stride) {
    const int i = c + (lane >> 4);
    const bool in = i < H / 8;
    u32x4_t a = rr[in ? i : H / 8 - 1], b = xr[in ? i : H / 8 - 1];
    if (!in) a = b = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t aw = a[q], bw = b[q];
      acc = __builtin_amdgcn_mfma_f64_16x16x4f64(lo_bf16(aw), lo_bf16(bw), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f64_16x16x4f64(hi_bf16(aw), hi_bf16(bw), acc, 0, 0, 0);
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave * 256 + v * 64 + lane] = acc[v];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  // Thread i: expert i % 16 of token i / 16.
  const int r = threadIdx.x & 15, c = threadIdx.x >> 4;
  const double* p = red + (r >> 2) * 64 + (r & 3) * 16 + c;
  double sum = p[0];
#pragma unroll
  for (int w = 1; w < kTileWaves; ++w) sum += p[w * 256];
  if (t0 + c < T && e0 + r < E)
    logits[((int64_t)blockIdx.z * T + t0 + c) * E + e0 + r] = sum;
}

template <int kPerLane, int kCount>
__global__ __launch_bounds__(64) void route_top_kernel(const double* __restrict__ logits, int T,
                                                       int E, int top_k, int renormalize,
                                                       int32_t* __restrict__ ids,
                                                       float* __restrict__ weights) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  double l[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    double v[kCount];
#pragma unroll
    for (int s = 0; s < kCount; ++s)
      v[s] = logits[((int64_t)s * T + t) * E + min(i * 64 + lane, E - 1)];
    l[i] = v[0];
#pragma unroll
    for (int s = 1; s < kCount; ++s) l[i] += v[s];
  }
  choose(l, E, top_k, renormalize, ids + t * top_k, weights + t * top_k);
}

template <int kCount>
hipError_t launch_top(const double* logits, int T, int E, int top_k, int renormalize, int32_t* ids,
                      float* weights, hipStream_t stream) {
  const auto kernel = E <= 64    ? route_top_kernel<1, kCount>
                      : E <= 128 ? route_top_kernel<2, kCount>
                      : E <= 256 ? route_top_kernel<4, kCount>
                                 : route_top_kernel<16, kCount>;
  hipLaunchKernelGGL(kernel, dim3(T), dim3(64), 0, stream, logits, T, E, top_k, renormalize, ids,
                     weights);
  return hipGetLastError();
}

// One workgroup a token does all of 64-bit arithmetic on one CU: up to 64 Ki
// products and a token a CU that is no slower than the tiles (51 tokens x 800,
// 87 experts, 70 Ki, 5.9 us against 6.2; 1 x 2240, 34 experts, 76 Ki, 7.2
// against 6.7; 14 x 1680, 128 experts, 215 Ki, 10.3 against 6.3; 512 tokens x
// 1024, 32 experts 8.9 against 7.6) and saves the host a launch. Past 128
// experts a wave's loads no longer fit its registers (2 tokens x 264, 180
// experts 8.0 us in one launch, 6.5 in two).
bool one_launch(int64_t T, int64_t H, int64_t E) {
  return E <= kOneMaxExperts && E * H <= 65536 && T <= 256;
}

// K's split over workgroups: the tiles are bound by 64-bit arithmetic, so up
// to a workgroup a CU (H = 4096: 32 tiles 18.8 us whole, 8.3 in 8 parts; 120
// tiles 18.9 whole, 12.9 in 2, 12.8 in 8; H = 1024: 32 tiles 9.5 and 7.4, 120
// tiles 9.6 whole, 8.2 in 2, 10.8 in 8).
int splits_of(int64_t T, int64_t E) {
  const int64_t tiles = ((T + kTile - 1) / kTile) * ((E + kTile - 1) / kTile);
  int splits = 1;
  while (splits < kMaxSplits && 2 * splits * tiles <= 256) splits *= 2;
  return splits;
}

}  // namespace

int64_t moe_route_workspace_bytes(int64_t T, int64_t H, int64_t E) {
  return one_launch(T, H, E) ? 0 : splits_of(T, E) * T * E * (int64_t)sizeof(double);
}

hipError_t launch_moe_route(const void* x, int64_t ldx, const void* router, int T, int H, int E,
                            int top_k, bool renormalize, int32_t* ids, float* weights,
                            double* logits, hipStream_t stream) {
  const auto* xb = static_cast<const uint8_t*>(x);
  const auto* rb = static_cast<const uint8_t*>(router);
  const int renorm = renormalize ? 1 : 0;
  if (one_launch(T, H, E)) {
    hipLaunchKernelGGL(E <= 64 ? route_one_kernel<1> : route_one_kernel<2>, dim3(T),
                       dim3(64 * kOneWaves), 0, stream, xb, ldx, rb, H, E, top_k, renorm, ids,
                       weights);
    return hipGetLastError();
  }
  const int splits = splits_of(T, E);
  hipLaunchKernelGGL(route_logits_kernel,
                     dim3((E + kTile - 1) / kTile, (T + kTile - 1) / kTile, splits),
                     dim3(64 * kTileWaves), 0, stream, xb, ldx, rb, T, H, E, logits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const auto top = splits == 1   ? launch_top<1>
                   : splits == 2 ? launch_top<2>
                   : splits == 4 ? launch_top<4>
                                 : launch_top<8>;
  return top(logits, T, E, top_k, renorm, ids, weights, stream);
}

}  // namespace mxfp4
