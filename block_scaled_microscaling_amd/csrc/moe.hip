// The experts of a mixture-of-experts layer for a few routed tokens, MXFP4
// weights, in two kernels.
//
// Mathematics, for pair p = t top_k + j with expert e = ids[p]:
//   a[p, i] = silu(sum_h Wg_e[i, h] x[t, h]) * (sum_h Wu_e[i, h] x[t, h])
//   y[t, h] = sum_j weights[t, j] sum_i W2_e[h, i] a[p, i]
// Weights are exact in BF16, sums and a are FP32. The second product takes a
// as FP32 (one token) or as the sum of BF16 pieces in columns of the same
// MFMA: three, all of FP32's significand, for FP32 results; two, 16 bits, for
// BF16 results, whose own rounding is 2^8 times larger.
//
// What bounds it: the chosen experts' weights, 3 H I 17/32 bytes each, read
// once: HBM.
//
// One token: as gemv's one-row kernel. The first kernel's workgroup has two
// gate and two up rows of a pair's expert; the second's four rows of y, over
// the blocks of all its experts in a row, so the sum over j needs no other
// workgroup. Several tokens: an expert's weights are read once for all its
// pairs, by few_stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

constexpr int kMaxWaves = 8;
constexpr int kOneDownRows = 8;
constexpr int kOneDownWaves = 7;  // 63 KiB of LDS
constexpr int kMaxPairs = 1024;
constexpr int kMaxExperts = 1024;
constexpr int kMapWords = kMaxExperts / 32;
constexpr int kMaxParts = kMoeMaxParts;

template <bool kOutFp32>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
  if constexpr (kOutFp32)
    static_cast<float*>(y)[at] = v;
  else
    static_cast<uint16_t*>(y)[at] = (uint16_t)pack_bf16x2(v, v);
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// --------------------------------------------------------------- one token
__global__ __launch_bounds__(64 * kMaxWaves) void moe_one_up_kernel(
    const uint8_t* __restrict__ x, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const uint8_t* __restrict__ w13_s, int HB, int I, int E,
    float* __restrict__ act) {
  __shared__ float red[kMaxWaves * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int e = ids[blockIdx.y];
  if (e < 0 || e >= E) return;
  const int64_t gate = (int64_t)e * 2 * I + 2 * blockIdx.x;
  const int64_t row[4] = {gate, gate + 1, gate + I, gate + I + 1};
  float acc[4] = {};
  for (int s = wave; s * 64 < HB; s += waves) {
    const bool in = s * 64 + lane < HB;
    const int b = in ? s * 64 + lane : HB - 1;
    u32x4_t w[4], xv[4];
    uint32_t byte[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[r] = *reinterpret_cast<const u32x4_t*>(w13 + row[r] * HB * 16 + (int64_t)b * 16);
      byte[r] = w13_s[row[r] * HB + b];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      xv[q] = *reinterpret_cast<const u32x4_t*>(x + (int64_t)b * 64 + 16 * q);
    if (!in) {
#pragma unroll
      for (int q = 0; q < 4; ++q) xv[q] = u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[r] = dot_block(w[r], scale_of_byte(in ? byte[r] : 127u), xv, acc[r]);
  }
  const float sum = sum_four_rows(acc);
  if ((lane & 15) == 0) red[wave * 4 + (lane >> 4)] = sum;
  __syncthreads();
  if (threadIdx.x < 2) {
    float g = red[threadIdx.x], u = red[2 + threadIdx.x];
    for (int w = 1; w < waves; ++w) {
      g += red[w * 4 + threadIdx.x];
      u += red[w * 4 + 2 + threadIdx.x];
    }
    act[(int64_t)blockIdx.y * I + 2 * blockIdx.x + threadIdx.x] = silu_mul(g, u);
  }
}

// Eight rows of y and not four: every workgroup reads all of the activations
// from L2 (8 experts, top 2, 4096 x 14336: 15.8 against 19.4 us, with the
// activations left out 14.7 us), as whole lines through the wave's LDS (a
// block's 128 bytes a lane straight from memory: 22.3 us with four rows).
template <bool kOutFp32>
__global__ __launch_bounds__(64 * kOneDownWaves) void moe_one_down_kernel(
    const float* __restrict__ act, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ w2_s, int H, int IB, int E, int top_k, void* __restrict__ y) {
  constexpr int R = kOneDownRows;
  using Blocks = LaneBlocks<8>;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ float red[kOneDownWaves * R];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  uint8_t* mine = lds + wave * Blocks::kBytes;
  const int h0 = blockIdx.x * R;
  const int blocks = top_k * IB;
  float acc[R / 4][4] = {};
  // Block b of pair j is the (j IB + b)-th; lanes without one, and those of
  // an absent expert, load no weights.
  for (int s = wave; s * 64 < blocks; s += waves) {
    const int at = s * 64 + lane;
    const int j = min(at, blocks - 1) / IB, b = at - j * IB;
    const int e = ids[j];
    const bool here = at < blocks && e >= 0 && e < E;
    u32x4_t w[R], a[8];
    uint32_t byte[R];
    float weight = 0.0f;
    if (here) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = (int64_t)e * H + h0 + r;
        w[r] = *reinterpret_cast<const u32x4_t*>(w2 + (row * IB + b) * 16);
        byte[r] = w2_s[row * IB + b];
      }
      weight = weights[j];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      a[q] = *reinterpret_cast<const u32x4_t*>(
          act + (int64_t)min(s * 512 + q * 64 + lane, blocks * 8 - 1) * 4);
    wave_sync();
    Blocks::fill(mine, a);
    if (here) {
#pragma unroll
      for (int q = 0; q < 8; ++q) a[q] = Blocks::get(mine, q);
#pragma unroll
      for (int r = 0; r < R; ++r)
        acc[r / 4][r % 4] = fmaf(weight, dot_block_f32(w[r], scale_of_byte(byte[r]), a),
                                 acc[r / 4][r % 4]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; r += 4) {
    const float sum = sum_four_rows(acc[r / 4]);
    if ((lane & 15) == 0) red[wave * R + r + (lane >> 4)] = sum;
  }
  __syncthreads();
  if (threadIdx.x < R) {
    float v = red[threadIdx.x];
    for (int w = 1; w < waves; ++w) v += red[w * R + threadIdx.x];
    store_y<kOutFp32>(y, h0 + threadIdx.x, v);
  }
}

// ------------------------------------------------------------ several tokens
// A wave writes the pairs of expert e in ascending order; returns how many.
__device__ __forceinline__ int list_pairs(const int32_t* ids, int pairs, int e, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  wave_sync();
#pragma unroll 4
  for (int base = 0; base < pairs; base += 64) {
    const int p = base + lane;
    const bool hit = ids[min(p, pairs - 1)] == e && p < pairs;
    const uint64_t m = __ballot(hit);
    if (hit) list[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)p;
    n += __popcll(m);
  }
  wave_sync();
  return n;
}

struct UpArgs {
  const uint8_t* x;
  int64_t ldx;
  const uint8_t* w13;
  const uint8_t* w13_s;
  float* act;
  int HB, I, top_k;
};

// 16 activation columns of pairs list[p0 .. p0 + 4 XL): the gate and the up
// rows are the two tiles of few_stream, K goes round the waves.
template <int XL>
__device__ __forceinline__ void up_tile(const UpArgs& g, int64_t gate, int i0,
                                        const uint16_t* list, int p0, int n, uint8_t* lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  BfRows<XL> rows;
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int p = list[min(p0 + 4 * i + (lane >> 4), n - 1)];
    rows.p[i] = g.x + (int64_t)(p / g.top_k) * g.ldx * 2 + (lane & 3) * 16;
  }
  const uint8_t* wc[2] = {g.w13 + gate * g.HB * 16, g.w13 + (gate + g.I) * g.HB * 16};
  const uint8_t* ws[2] = {g.w13_s + gate * g.HB, g.w13_s + (gate + g.I) * g.HB};
  v4f_t acc[2] = {v4f_t{}, v4f_t{}};
  few_stream<2>(wc, ws, [](int, int r) { return r; }, rows, g.HB, wave, waves,
                lds + wave * few_lds_bytes<2, BfRows<XL>>(), acc);
  __syncthreads();
  auto* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[(t * waves + wave) * 256 + v * 64 + lane] = acc[t][v];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * XL; i += blockDim.x) {
    const int r = i & 15, c = i >> 4;
    const float* part = red + (r & 3) * 64 + (r >> 2) * 16 + c;
    float gv = part[0], uv = part[waves * 256];
    for (int w = 1; w < waves; ++w) {
      gv += part[w * 256];
      uv += part[(waves + w) * 256];
    }
    if (p0 + c < n) g.act[(int64_t)list[p0 + c] * g.I + i0 + r] = silu_mul(gv, uv);
  }
  __syncthreads();
}

// One workgroup per 16 activation columns and expert. With fewer pairs than
// experts the grid counts pairs, and the first pair of an expert stands for
// all of its pairs. Also clears what the second kernel counts with.
template <int kMaxXL>
__global__ __launch_bounds__(64 * kMaxWaves) void moe_up_kernel(
    UpArgs g, const int32_t* __restrict__ ids, int pairs, int E, int by_pair, uint32_t* counters,
    int n_counters) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t list[kMaxPairs];
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < n_counters; i += blockDim.x) counters[i] = 0;
  const int e = by_pair ? ids[blockIdx.y] : (int)blockIdx.y;
  if (e < 0 || e >= E) return;
  // Every wave writes the same list.
  const int n = list_pairs(ids, pairs, e, list);
  if (n == 0 || (by_pair && list[0] != blockIdx.y)) return;
  const int i0 = blockIdx.x * kFewTile;
  const int64_t gate = (int64_t)e * 2 * g.I + i0;
  for (int p0 = 0; p0 < n; p0 += 4 * kMaxXL) {
    const int left = n - p0;
    if (left <= 4)
      up_tile<1>(g, gate, i0, list, p0, n, lds);
    else if (kMaxXL == 2 || left <= 8)
      up_tile<2>(g, gate, i0, list, p0, n, lds);
    else
      up_tile<kMaxXL>(g, gate, i0, list, p0, n, lds);
  }
}

// The chosen experts as a bit map, and the pairs' experts (-1: absent).
__device__ __forceinline__ void read_chosen(const int32_t* __restrict__ ids, int pairs, int E,
                                            int32_t* chosen, uint32_t* map) {
  if (threadIdx.x < kMapWords) map[threadIdx.x] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    const int e = ids[p];
    const bool here = e >= 0 && e < E;
    chosen[p] = here ? e : -1;
    if (here) atomicOr(&map[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// The n-th chosen expert (from 0) in order of its index, of more than n.
__device__ __forceinline__ int nth_chosen(const uint32_t* map, int n) {
  int w = 0;
  for (; n >= __popc(map[w]); ++w) n -= __popc(map[w]);
  uint32_t m = map[w];
  for (int i = 0; i < n; ++i) m &= m - 1;
  return w * 32 + __ffs(m) - 1;
}

// One workgroup per 16 outputs h and part of the chosen experts (every
// gridDim.y-th). Its waves take the experts in turn, with few experts also
// the units of K; the pairs' results stay in LDS and are summed in order of
// j. The last workgroup of an h to finish adds the parts, in order of part,
// so y is the same on every run.
template <int kRows, int kPieces, bool kOutFp32>
__global__ __launch_bounds__(64 * kMaxWaves) void moe_down_kernel(
    const float* __restrict__ act, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ w2_s, int T, int H, int I, int E, int top_k, int max_split,
    float* __restrict__ partial, uint32_t* __restrict__ counters, void* __restrict__ y) {
  using X = F32Rows<kRows, kPieces>;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint32_t map[kMapWords];
  __shared__ uint32_t arrived;
  const int pairs = T * top_k;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  auto* part = reinterpret_cast<float*>(lds + waves * few_lds_bytes<1, X>());  // [split][pair][16]
  auto* chosen = reinterpret_cast<int32_t*>(part + max_split * pairs * 16);
  auto* list = reinterpret_cast<uint16_t*>(chosen + pairs) + wave * pairs;
  read_chosen(ids, pairs, E, chosen, map);
  int experts = 0;
  for (int w = 0; w < (E + 31) / 32; ++w) experts += __popc(map[w]);
  const int parts = gridDim.y, mine = blockIdx.y;
  const int held = (experts - mine + parts - 1) / parts;  // experts of this part
  const int h0 = blockIdx.x * kFewTile;
  const int IB = I / 32;
  int split = 1;
  while (2 * split <= max_split && 2 * split * held <= waves) split *= 2;
  for (int item = wave; item < held * split; item += waves) {
    const int s = item % split;
    const int e = __builtin_amdgcn_readfirstlane(nth_chosen(map, item / split * parts + mine));
    const int n = list_pairs(chosen, pairs, e, list);
    const int64_t row = (int64_t)e * H + h0;
    const uint8_t* wc[1] = {w2 + row * IB * 16};
    const uint8_t* ws[1] = {w2_s + row * IB};
    for (int p0 = 0; p0 < n; p0 += kRows) {
      X rows;
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i)
        rows.p[i] =
            act + (int64_t)list[min(p0 + 2 * i + (lane >> 5), n - 1)] * I + (lane & 7) * 4;
      v4f_t acc[1] = {v4f_t{}};
      few_stream<1>(wc, ws, [](int, int r) { return r; }, rows, IB, s, split,
                    lds + wave * few_lds_bytes<1, X>(), acc);
      const int c = lane & 15;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        // Sum of the pieces' columns.
        float sum = c < X::kColumns ? acc[0][v] : 0.0f;
        sum += __shfl_xor(sum, kRows);
        if (kPieces == 3) sum += __shfl_xor(sum, 2 * kRows);
        if (c < kRows && p0 + c < n)
          part[(s * pairs + list[p0 + c]) * 16 + 4 * (lane >> 4) + v] = sum;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * 16; i += blockDim.x) {
    const int t = i >> 4, r = i & 15;
    float sum = 0.0f;
    for (int j = 0; j < top_k; ++j) {
      const int p = t * top_k + j, e = chosen[p];
      if (e < 0) continue;
      if (parts > 1) {
        int rank = __popc(map[e >> 5] & ((1u << (e & 31)) - 1));
        for (int w = 0; w < e >> 5; ++w) rank += __popc(map[w]);
        if (rank % parts != mine) continue;
      }
      float v = part[p * 16 + r];
      for (int s = 1; s < split; ++s) v += part[(s * pairs + p) * 16 + r];
      sum += weights[p] * v;
    }
    if (parts == 1)
      store_y<kOutFp32>(y, (int64_t)t * H + h0 + r, sum);
    else
      __hip_atomic_store(&partial[((int64_t)mine * T + t) * H + h0 + r], sum, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
  }
  if (parts == 1) return;
  // The parts go through memory as device-scope atomics, which no XCD's L2
  // holds back, and a wave's are complete once its count of outstanding
  // stores is zero: so the workgroup counts as arrived after its stores, and
  // the last one reads all of them. (Ordinary stores with a release fence
  // write back a whole L2 in every workgroup: 7 tokens, H 1056, I 544, 10
  // experts took 56 us instead of 15.)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(&counters[blockIdx.x], 1u, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived != (uint32_t)parts - 1) return;
  for (int i = threadIdx.x; i < T * 16; i += blockDim.x) {
    const int64_t at = (int64_t)(i >> 4) * H + h0 + (i & 15);
    float sum = 0.0f;
    for (int s = 0; s < parts; ++s)
      sum += __hip_atomic_load(&partial[(int64_t)s * T * H + at], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    store_y<kOutFp32>(y, at, sum);
  }
}

template <int kMaxXL>
hipError_t launch_up(const UpArgs& g, const int32_t* ids, int pairs, int E, uint32_t* counters,
                     int n_counters, hipStream_t stream) {
  const int waves = even_waves((g.HB + kUnitBlocks - 1) / kUnitBlocks, 4);
  const int lds = waves * few_lds_bytes<2, BfRows<kMaxXL>>();
  hipLaunchKernelGGL((moe_up_kernel<kMaxXL>), dim3(g.I / kFewTile, pairs < E ? pairs : E),
                     dim3(64 * waves), lds, stream, g, ids, pairs, E, pairs < E ? 1 : 0, counters,
                     n_counters);
  return hipGetLastError();
}

template <int kRows, int kPieces, bool kOutFp32>
hipError_t launch_down(const float* act, const int32_t* ids, const float* weights,
                       const uint8_t* w2, const uint8_t* w2_s, int T, int H, int I, int E,
                       int top_k, int parts, int max_split, float* partial, uint32_t* counters,
                       void* y, hipStream_t stream) {
  const int pairs = T * top_k, waves = kMaxWaves;
  const int lds = waves * few_lds_bytes<1, F32Rows<kRows, kPieces>>() + max_split * pairs * 64 +
                  pairs * 4 + waves * pairs * 2;
  const auto kernel = moe_down_kernel<kRows, kPieces, kOutFp32>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3(H / kFewTile, parts), dim3(64 * waves), lds, stream, act, ids,
                     weights, w2, w2_s, T, H, I, E, top_k, max_split, partial, counters, y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(const void* x, int64_t ldx, const int32_t* ids, const float* weights,
                      const void* w13, const void* w13_s, const void* w2, const void* w2_s, int T,
                      int H, int I, int E, int top_k, bool out_fp32, void* y, void* workspace,
                      hipStream_t stream) {
  const auto* xb = static_cast<const uint8_t*>(x);
  const auto* c13 = static_cast<const uint8_t*>(w13);
  const auto* s13 = static_cast<const uint8_t*>(w13_s);
  const auto* c2 = static_cast<const uint8_t*>(w2);
  const auto* s2 = static_cast<const uint8_t*>(w2_s);
  const int pairs = T * top_k, HB = H / 32, IB = I / 32;
  // Workspace: partial sums of y, the activations, the counters.
  auto* partial = static_cast<float*>(workspace);
  auto* act = partial + (T > 1 ? (int64_t)kMaxParts * T * H : 0);
  auto* counters = reinterpret_cast<uint32_t*>(act + (int64_t)pairs * I);
  hipError_t e;
  if (T == 1) {
    hipLaunchKernelGGL(moe_one_up_kernel, dim3(I / 2, top_k),
                       dim3(64 * even_waves((HB + 63) / 64, kMaxWaves)), 0, stream, xb, ids, c13,
                       s13, HB, I, E, act);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 threads(64 * even_waves((top_k * IB + 63) / 64, kOneDownWaves));
    hipLaunchKernelGGL(out_fp32 ? moe_one_down_kernel<true> : moe_one_down_kernel<false>,
                       dim3(H / kOneDownRows), threads, threads.x / 64 * LaneBlocks<8>::kBytes, stream, act, ids, weights, c2, s2, H, IB, E, top_k,
                       y);
    return hipGetLastError();
  }
  const int chosen = pairs < E ? pairs : E;  // experts, at most
  const UpArgs up = {xb, ldx, c13, s13, act, HB, I, top_k};
  e = pairs > 6 * E ? launch_up<4>(up, ids, pairs, E, counters, H / kFewTile, stream)
                    : launch_up<2>(up, ids, pairs, E, counters, H / kFewTile, stream);
  if (e != hipSuccess) return e;
  int parts = (512 + H / kFewTile - 1) / (H / kFewTile);
  if (parts > kMaxParts) parts = kMaxParts;
  if (parts > chosen) parts = chosen;
  int max_split = 1;
  while (2 * max_split * chosen <= kMaxWaves * parts && 2 * max_split * pairs <= kMaxPairs)
    max_split *= 2;
  if (out_fp32)
    return launch_down<4, 3, true>(act, ids, weights, c2, s2, T, H, I, E, top_k, parts, max_split,
                                   partial, counters, y, stream);
  if (pairs > 4 * E)
    return launch_down<8, 2, false>(act, ids, weights, c2, s2, T, H, I, E, top_k, parts,
                                    max_split, partial, counters, y, stream);
  return launch_down<4, 2, false>(act, ids, weights, c2, s2, T, H, I, E, top_k, parts, max_split,
                                  partial, counters, y, stream);
}

}  // namespace mxfp4
