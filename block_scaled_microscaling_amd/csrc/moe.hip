// The experts of a mixture-of-experts layer for a few routed tokens, MXFP4
// weights, in two kernels.
//
// Mathematics, for pair p = t top_k + j with expert e = ids[p]:
//   a[p, i] = silu(sum_h Wg_e[i, h] x[t, h]) * (sum_h Wu_e[i, h] x[t, h])
//   y[t, h] = sum_j weights[t, j] sum_i W2_e[h, i] a[p, i]
// Weights are exact in BF16 and sums are FP32. a is handed to the second
// product as hi + lo, both BF16 (hi = a rounded, lo = a - hi rounded): 16
// significand bits, so that y's error stays that of its FP32 sums and one
// rounding to its type. The two halves ride in different columns of the same
// MFMA (8 pairs a time), so lo costs no further weight reads or MFMAs.
//
// What bounds it: the chosen experts' weights, 3 H I 17/32 bytes each, read
// once: HBM.
//
// Work split. First kernel: one workgroup per 16 activation columns and
// place in the list of chosen experts; K chunks go round its 8 waves. Second
// kernel: one workgroup per 16 outputs h and all pairs, whose results stay
// in LDS: its waves take the chosen experts in turn, and the sum over j runs
// in order of j, so y is the same on every run.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxPairs = 1024;
constexpr int kMaxExperts = 1024;
constexpr int kMapWords = kMaxExperts / 32;
constexpr int kLdsSlots = 1024;  // pair results held at once, 16 outputs each

constexpr int kFewChunkBlocks = 8;  // 32-element blocks a wave takes per step (256 k)

// Adds the product over the K chunks c0, c0 + cs, ... of KB blocks to acc
// for kRT row tiles that share the token rows. codes[i], scales[i]: the
// lane's row of tile i; x: the lane's token row; g: the lane's K group.
template <int kRT>
__device__ __forceinline__ void few_mac(const uint8_t* const (&codes)[kRT],
                                        const uint8_t* const (&scales)[kRT], const uint8_t* x,
                                        int KB, int c0, int cs, int g, v4f_t (&acc)[kRT]) {
  const int chunks = (KB + kFewChunkBlocks - 1) / kFewChunkBlocks;
  for (int c = c0; c < chunks; c += cs) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // Blocks past the row are read as block KB - 1 and count as zeros on
      // both sides.
      const int b = c * kFewChunkBlocks + 2 * g + j;
      const bool in = b < KB;
      const int bb = in ? b : KB - 1;
      u32x4_t w[kRT], xv[4];
      float s[kRT];
#pragma unroll
      for (int i = 0; i < kRT; ++i) {
        w[i] = *reinterpret_cast<const u32x4_t*>(codes[i] + (int64_t)bb * 16);
        s[i] = scale_of_byte(scales[i][bb]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        xv[q] = *reinterpret_cast<const u32x4_t*>(x + (int64_t)bb * 64 + 16 * q);
      if (!in) {
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
          w[i] = u32x4_t{0u, 0u, 0u, 0u};
          s[i] = 1.0f;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) xv[q] = u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bf16x8_t xb = __builtin_bit_cast(bf16x8_t, xv[q]);
#pragma unroll
        for (int i = 0; i < kRT; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(w[i][q], s[i]), xb, acc[i], 0,
                                                           0, 0);
      }
    }
  }
}

// The pairs and which experts they chose, in LDS.
struct Chosen {
  int32_t ids[kMaxPairs];
  uint32_t map[kMapWords];  // bit e: some pair chose expert e
};

__device__ __forceinline__ void read_chosen(Chosen& c, const int32_t* __restrict__ ids, int pairs,
                                            int E) {
  if (threadIdx.x < kMapWords) c.map[threadIdx.x] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += kThreads) {
    const int e = ids[p];
    const bool here = e >= 0 && e < E;
    c.ids[p] = here ? e : -1;
    if (here) atomicOr(&c.map[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// The n-th chosen expert (from 0) in order of its index, or -1.
__device__ __forceinline__ int nth_chosen(const Chosen& c, int n, int E) {
  const int words = (E + 31) / 32;
  for (int w = 0; w < words; ++w) {
    uint32_t m = c.map[w];
    const int count = __popc(m);
    if (n < count) {
      for (int i = 0; i < n; ++i) m &= m - 1;
      return w * 32 + __ffs(m) - 1;
    }
    n -= count;
  }
  return -1;
}

__device__ __forceinline__ int count_chosen(const Chosen& c, int E) {
  int n = 0;
  for (int w = 0; w < (E + 31) / 32; ++w) n += __popc(c.map[w]);
  return n;
}

// One wave writes the pairs of expert e in ascending order; returns how many.
__device__ __forceinline__ int list_pairs(const Chosen& c, int pairs, int e, int lane,
                                          uint16_t* list) {
  int n = 0;
  wave_sync();
  for (int base = 0; base < pairs; base += 64) {
    const int p = base + lane;
    const bool hit = p < pairs && c.ids[p] == e;
    const uint64_t m = __ballot(hit);
    if (hit) list[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)p;
    n += __popcll(m);
  }
  wave_sync();
  return n;
}

__global__ __launch_bounds__(kThreads) void moe_up_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const uint8_t* __restrict__ w13_s, int pairs, int H, int I,
    int E, int top_k, uint16_t* __restrict__ act) {
  __shared__ Chosen chosen;
  __shared__ uint16_t list[kMaxPairs];
  __shared__ int count;
  __shared__ __align__(16) float red[2 * kWaves * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  read_chosen(chosen, ids, pairs, E);
  const int e = nth_chosen(chosen, blockIdx.y, E);
  if (e < 0) return;
  if (wave == 0) {
    const int n = list_pairs(chosen, pairs, e, lane, list);
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int n_pairs = count;
  const int i0 = blockIdx.x * kFewTile;
  const int HB = H / 32;
  const int64_t gate = (int64_t)e * 2 * I + i0 + (lane & 15);
  const uint8_t* wc[2] = {w13 + gate * HB * 16, w13 + (gate + I) * HB * 16};
  const uint8_t* ws[2] = {w13_s + gate * HB, w13_s + (gate + I) * HB};
  for (int p0 = 0; p0 < n_pairs; p0 += kFewTile) {
    const int mine = list[min(p0 + (lane & 15), n_pairs - 1)];
    v4f_t acc[2] = {v4f_t{}, v4f_t{}};
    few_mac<2>(wc, ws, x + (int64_t)(mine / top_k) * ldx * 2, HB, wave, kWaves, lane >> 4, acc);
    if (p0 > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[(i * kWaves + wave) * 256 + v * 64 + lane] = acc[i][v];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
      const int at = (r & 3) * 64 + (r >> 2) * 16 + t;
      float g = red[at], u = red[kWaves * 256 + at];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        g += red[w * 256 + at];
        u += red[(kWaves + w) * 256 + at];
      }
      if (p0 + t < n_pairs) {
        const float a = g / (1.0f + expf(-g)) * u;
        const uint32_t hi = pack_bf16x2(a, a) & 0xFFFFu;
        // lo is 0 where hi is no finite number: inf - inf would make it NaN.
        const float rest = (hi & 0x7F80u) == 0x7F80u ? 0.0f : a - __uint_as_float(hi << 16);
        uint16_t* o = act + (int64_t)list[p0 + t] * 2 * I + i0 + r;
        o[0] = (uint16_t)hi;
        o[I] = (uint16_t)pack_bf16x2(rest, rest);
      }
    }
  }
}

template <bool kOutFp32>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(
    const uint16_t* __restrict__ act, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ w2_s, int T, int H, int I, int E, int top_k, int max_split,
    void* __restrict__ y) {
  extern __shared__ __align__(16) float part[];  // [split][pair][16]
  __shared__ Chosen chosen;
  __shared__ uint16_t lists[kWaves][kMaxPairs];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int pairs = T * top_k;
  read_chosen(chosen, ids, pairs, E);
  const int experts = count_chosen(chosen, E);
  // With fewer experts than waves the K chunks of each go round `split` waves.
  int split = 1;
  while (2 * split <= max_split && 2 * split * experts <= kWaves) split *= 2;
  const int h0 = blockIdx.x * kFewTile;
  const int IB = I / 32;
  for (int item = wave; item < experts * split; item += kWaves) {
    const int s = item % split;
    const int e = nth_chosen(chosen, item / split, E);
    const int n_pairs = list_pairs(chosen, pairs, e, lane, lists[wave]);
    const int64_t row = (int64_t)e * H + h0 + (lane & 15);
    const uint8_t* wc[1] = {w2 + row * IB * 16};
    const uint8_t* ws[1] = {w2_s + row * IB};
    // Columns 0..7: hi of 8 pairs; columns 8..15: lo of the same.
    for (int p0 = 0; p0 < n_pairs; p0 += 8) {
      const int mine = lists[wave][min(p0 + (lane & 7), n_pairs - 1)];
      const uint16_t* a = act + ((int64_t)mine * 2 + ((lane >> 3) & 1)) * I;
      v4f_t acc[1] = {v4f_t{}};
      few_mac<1>(wc, ws, reinterpret_cast<const uint8_t*>(a), IB, s, split, lane >> 4, acc);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float sum = acc[0][v] + __shfl_xor(acc[0][v], 8);
        if ((lane & 8) == 0 && p0 + (lane & 7) < n_pairs)
          part[((int64_t)s * pairs + mine) * 16 + 4 * (lane >> 4) + v] = sum;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * 16; i += kThreads) {
    const int t = i >> 4, r = i & 15;
    float sum = 0.0f;
    for (int j = 0; j < top_k; ++j) {
      const int p = t * top_k + j;
      if (chosen.ids[p] < 0) continue;
      float v = part[p * 16 + r];
      for (int s = 1; s < split; ++s) v += part[(s * pairs + p) * 16 + r];
      sum += weights[p] * v;
    }
    const int64_t o = (int64_t)t * H + h0 + r;
    if constexpr (kOutFp32)
      static_cast<float*>(y)[o] = sum;
    else
      static_cast<uint16_t*>(y)[o] = (uint16_t)pack_bf16x2(sum, sum);
  }
}

}  // namespace

hipError_t launch_moe(const void* x, int64_t ldx, const int32_t* ids, const float* weights,
                      const void* w13, const void* w13_s, const void* w2, const void* w2_s, int T,
                      int H, int I, int E, int top_k, bool out_fp32, void* y, uint16_t* act,
                      hipStream_t stream) {
  const int pairs = T * top_k;
  hipLaunchKernelGGL(moe_up_kernel, dim3(I / kFewTile, pairs < E ? pairs : E), dim3(kThreads), 0,
                     stream, static_cast<const uint8_t*>(x), ldx, ids,
                     static_cast<const uint8_t*>(w13), static_cast<const uint8_t*>(w13_s), pairs,
                     H, I, E, top_k, act);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  int max_split = kWaves;
  while (max_split > 1 && max_split * pairs > kLdsSlots) max_split /= 2;
  const size_t lds = (size_t)max_split * pairs * 16 * sizeof(float);
  const auto kernel = out_fp32 ? moe_down_kernel<true> : moe_down_kernel<false>;
  err = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(kernel, dim3(H / kFewTile), dim3(kThreads), lds, stream, act, ids, weights,
                     static_cast<const uint8_t*>(w2), static_cast<const uint8_t*>(w2_s), T, H, I,
                     E, top_k, max_split, y);
  return hipGetLastError();
}

}  // namespace mxfp4
