// The experts of a mixture-of-experts layer for a few routed tokens, MXFP4
// weights.
//
// Mathematics, for pair p = t top_k + j with expert e = ids[p]:
//   a[p, i] = silu(sum_h Wg_e[i, h] x[t, h]) * (sum_h Wu_e[i, h] x[t, h])
//   y[t, h] = sum_j weights[t, j] sum_i W2_e[h, i] a[p, i]
// Weights are exact in BF16, sums and a are FP32. The second product takes a
// as FP32 (by pairs) or as the sum of three BF16 pieces, all of FP32's
// significand, in columns of the same MFMA, so that a token's precision does
// not depend on which of the two the batch beside it takes. Two pieces, 16 bits,
// are 5 to 20% faster but change 0.2% of BF16 results by a step, and all that
// is left of large activations that cancel. The first kernel by experts writes
// the pieces, so that they are made once.
//
// What bounds it: the chosen experts' weights, 3 H I 17/32 bytes each, read
// once: HBM (1 token through 2 of 8 experts of 4096 x 14336, 187 MB, 22 + 16
// us; 32 tokens through 112 of 128 of 2048 x 768, 281 MB, 73 us), or
// latency where they are few (1 token through 8 of the latter, 4.9 + 4.8 us).
//
// Few pairs: as gemv's one-row kernel, in two launches. The first kernel's
// workgroup has two gate and two up rows of a pair's expert; the second's
// eight rows of a token's y, over the blocks of all its experts one after the
// other, so the sum over j needs no other workgroup. Many pairs: an expert's
// weights are read once for all its pairs, by few_stream (W2 by share_stream
// where an expert has many), and a third launch sums the pairs' parts of y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

constexpr int kPairDownRows = 8;
constexpr int kPairDownWaves = 7;  // 63 KiB of LDS
constexpr int kTileWaves = 4;   // of the kernels for several tokens
constexpr int kDenseParts = 2;  // parts of K of the kernel for many pairs an expert
constexpr int kPieces = 3;      // BF16 pieces of an activation
constexpr int kDownRows = 4;    // pairs of the second kernel by experts: 12 columns

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// --------------------------------------------------------------- by pairs
__global__ __launch_bounds__(64 * kMaxWaves) void moe_pair_up_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const uint8_t* __restrict__ w13_s, int HB, int I, int E,
    int top_k, float* __restrict__ act) {
  __shared__ float red[kMaxWaves * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int e = ids[blockIdx.y];
  if (e < 0 || e >= E) return;
  x += blockIdx.y / top_k * ldx * 2;
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

// The same for H <= 32 kLanes: 128 / kLanes activation columns a wave. The
// call, before and now: 3 tokens x 288 x 7392, 22 experts, top 3, 17.7 -> 10.1
// us, 4 x 736 x 992, 82 top 4, 11.5 -> 9.5, 1 x 1120 x 11680, 5 top 2, 15.9 ->
// 14.8; with H of two segments it made no difference.
template <int kLanes>
__global__ __launch_bounds__(64 * kShortWaves) void moe_pair_up_short_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ w13, const uint8_t* __restrict__ w13_s, int HB, int I, int E,
    int top_k, float* __restrict__ act) {
  constexpr int kGroups = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int e = ids[blockIdx.y];
  if (e < 0 || e >= E) return;
  x += blockIdx.y / top_k * ldx * 2;
  const int i0 = (blockIdx.x * kShortWaves + wave) * 2 * kGroups;
  const int64_t gate = (int64_t)e * 2 * I + i0;
  w13 += gate * HB * 16;
  w13_s += gate * HB;
  // The lane's rows: columns j and kGroups + j, gate and up.
  const uint32_t j = lane / kLanes;
  const uint32_t row[4] = {j, kGroups + j, I + j, I + kGroups + j};
  const bool in = lane % kLanes < HB;
  const uint32_t b = in ? lane % kLanes : HB - 1;
  u32x4_t w[4], xv[4];
  uint32_t byte[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    w[r] = *reinterpret_cast<const u32x4_t*>(w13 + (row[r] * HB + b) * 16);
    byte[r] = w13_s[row[r] * HB + b];
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    xv[q] = *reinterpret_cast<const u32x4_t*>(x + b * 64 + 16 * q);
  if (!in) {
#pragma unroll
    for (int q = 0; q < 4; ++q) xv[q] = u32x4_t{0u, 0u, 0u, 0u};
  }
  float v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    v[r] = dot_block(w[r], scale_of_byte(in ? byte[r] : 127u), xv, 0.0f);
  act += (int64_t)blockIdx.y * I + i0 + j;
  if constexpr (kLanes == 64) {
    const float s = sum_four_rows(v), up = __shfl_xor(s, 32);
    if ((lane & 15) == 0 && lane < 32) act[lane >> 4] = silu_mul(s, up);
  } else if constexpr (kLanes == 32) {
    // Even 16 lanes: the first columns, odd ones: the second.
    const float a = silu_mul(sum16(merge16(v[0], v[1])), sum16(merge16(v[2], v[3])));
    if ((lane & 15) == 0) act[((lane >> 4) & 1) * kGroups] = a;
  } else {
    const bool second = lane & 1;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = sum16(v[r]);
    const float a = silu_mul(second ? v[1] : v[0], second ? v[3] : v[2]);
    if ((lane & 15) < 2) act[(lane & 1) * kGroups] = a;
  }
}

// Eight rows of y and not four: every workgroup reads all of the activations
// from L2 (8 experts, top 2, 4096 x 14336: 15.8 against 19.4 us, with the
// activations left out 14.7 us), as whole lines through the wave's LDS (a
// block's 128 bytes a lane straight from memory: 22.3 us with four rows).
template <bool kOutFp32>
__global__ __launch_bounds__(64 * kPairDownWaves) void moe_pair_down_kernel(
    const float* __restrict__ act, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, const uint8_t* __restrict__ w2,
    const uint8_t* __restrict__ w2_s, int H, int IB, int E, int top_k, void* __restrict__ y) {
  constexpr int R = kPairDownRows;
  using Blocks = LaneBlocks<8>;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ float red[kPairDownWaves * R];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  uint8_t* mine = lds + wave * Blocks::kBytes;
  const int h0 = blockIdx.x * R;
  const int blocks = top_k * IB;
  const int64_t t = blockIdx.y;
  act += t * blocks * 32;
  ids += t * top_k;
  weights += t * top_k;
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
    store_y<kOutFp32>(y, t * H + h0 + threadIdx.x, v);
  }
}

// -------------------------------------------------------------- by experts
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

// Products of two tiles of 16 weight rows, at the uniform rows row0 and row1,
// with X's columns, K split over the workgroup's waves; the results are left
// in LDS, for tile_sum.
template <class X>
__device__ __forceinline__ void two_tiles(const uint8_t* codes, const uint8_t* scales,
                                          int64_t row0, int64_t row1, int KB, const X& rows,
                                          uint8_t* lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const uint8_t* wc[2] = {codes + row0 * KB * 16, codes + row1 * KB * 16};
  const uint8_t* ws[2] = {scales + row0 * KB, scales + row1 * KB};
  v4f_t acc[2] = {v4f_t{}, v4f_t{}};
  __syncthreads();  // the last tiles' results have been read
  few_stream<2, true>(wc, ws, [](int, int r) { return r; }, rows, KB, wave, waves,
                lds + wave * few_lds_bytes<2, X>(), acc);
  __syncthreads();
  auto* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[(t * waves + wave) * 256 + v * 64 + lane] = acc[t][v];
  __syncthreads();
}

// Row r and column c of tile t of two_tiles' products.
__device__ __forceinline__ float tile_sum(const uint8_t* lds, int t, int r, int c) {
  const int waves = blockDim.x >> 6;
  const float* p = reinterpret_cast<const float*>(lds) + t * waves * 256 + (r & 3) * 64 +
                   (r >> 2) * 16 + c;
  float sum = p[0];
  for (int w = 1; w < waves; ++w) sum += p[w * 256];
  return sum;
}

struct UpArgs {
  const uint8_t* x;
  int64_t ldx;
  const uint8_t* w13;
  const uint8_t* w13_s;
  uint16_t* act;  // [pairs][I / 16][kPieces][16]: BF16 pieces of the activations
  int HB, I, top_k;
};

// The tokens of the pairs list[p0 .. p0 + 4 XL); past the n-th, of the last.
template <int XL>
__device__ __forceinline__ BfRows<XL> up_rows(const UpArgs& g, const uint16_t* list, int p0,
                                              int n) {
  const int lane = threadIdx.x & 63;
  BfRows<XL> rows;
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int p = list[min(p0 + 4 * i + (lane >> 4), n - 1)];
    rows.p[i] = g.x + (int64_t)(p / g.top_k) * g.ldx * 2 + (lane & 3) * 16;
  }
  return rows;
}

// Activations i0 .. i0 + 15 of the pairs list[p0 .. p0 + 4 XL), K split over
// the waves.
template <int XL>
__device__ __forceinline__ void up_tile(const UpArgs& g, int64_t gate, int i0,
                                        const uint16_t* list, int p0, int n, uint8_t* lds) {
  two_tiles(g.w13, g.w13_s, gate, gate + g.I, g.HB, up_rows<XL>(g, list, p0, n), lds);
  for (int i = threadIdx.x; i < 32 * XL; i += blockDim.x) {
    const int r = 2 * (i & 7), c = i >> 3;
    if (p0 + c >= n) continue;
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      v[j] = silu_mul(tile_sum(lds, 0, r + j, c), tile_sum(lds, 1, r + j, c));
    uint16_t* at = g.act + ((int64_t)list[p0 + c] * g.I + i0) * kPieces + r;
#pragma unroll
    for (int piece = 0; piece < kPieces; ++piece, at += kFewTile) {
      const uint32_t low = next_piece(v[0]);
      *reinterpret_cast<uint32_t*>(at) = low | (uint32_t)next_piece(v[1]) << 16;
    }
  }
}

// The same with a tile a wave, over all of H: no wave waits for another.
template <int XL>
__device__ __forceinline__ void up_wave(const UpArgs& g, int64_t gate, int i0,
                                        const uint16_t* list, int p0, int n, uint8_t* lds) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  const BfRows<XL> rows = up_rows<XL>(g, list, p0, n);
  const uint8_t* wc[2] = {g.w13 + gate * g.HB * 16, g.w13 + (gate + g.I) * g.HB * 16};
  const uint8_t* ws[2] = {g.w13_s + gate * g.HB, g.w13_s + (gate + g.I) * g.HB};
  v4f_t acc[2] = {v4f_t{}, v4f_t{}};
  few_stream<2, true>(wc, ws, [](int, int r) { return r; }, rows, g.HB, 0, 1, lds, acc);
  if (c >= 4 * XL || p0 + c >= n) return;
  v4f_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = silu_mul(acc[0][i], acc[1][i]);
  uint16_t* at = g.act + ((int64_t)list[p0 + c] * g.I + i0) * kPieces + 4 * (lane >> 4);
#pragma unroll
  for (int piece = 0; piece < kPieces; ++piece, at += kFewTile) {
    uint16_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f = v[i];
      b[i] = next_piece(f);
      v[i] = f;
    }
    *reinterpret_cast<uint2*>(at) = make_uint2(b[0] | (uint32_t)b[1] << 16,
                                               b[2] | (uint32_t)b[3] << 16);
  }
}

// A workgroup takes 16 activation columns of an expert, or, with kWaveTiles,
// each of its waves does.
template <int kMaxXL, bool kWaveTiles>
__global__ __launch_bounds__(64 * kTileWaves) void moe_up_kernel(
    UpArgs g, const int32_t* __restrict__ ids, int pairs) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t list[kMaxPairs];
  const int e = blockIdx.y;
  const int n = list_pairs(ids, pairs, e, list);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i0 = (kWaveTiles ? blockIdx.x * kTileWaves + wave : blockIdx.x) * kFewTile;
  if (n == 0 || i0 >= g.I) return;
  const int64_t gate = (int64_t)e * 2 * g.I + i0;
  uint8_t* mine = lds + wave * few_lds_bytes<2, BfRows<kMaxXL>>();
  const auto take = [&](auto xl, int p0) {
    constexpr int XL = decltype(xl)::value;
    if constexpr (kWaveTiles)
      up_wave<XL>(g, gate, i0, list, p0, n, mine);
    else
      up_tile<XL>(g, gate, i0, list, p0, n, lds);
  };
  for (int p0 = blockIdx.z * 4 * kMaxXL; p0 < n; p0 += gridDim.z * 4 * kMaxXL) {
    const int left = n - p0;
    if (left <= 4)
      take(std::integral_constant<int, 1>{}, p0);
    else if (kMaxXL == 2 || left <= 8)
      take(std::integral_constant<int, 2>{}, p0);
    else
      take(std::integral_constant<int, kMaxXL>{}, p0);
  }
}

struct DownArgs {
  const uint16_t* act;
  const uint8_t* w2;
  const uint8_t* w2_s;
  float* part;  // [pairs][H]: W2 a of each pair
  int H, I;
};

// The lane's place in the first block of a pair's piece.
__device__ __forceinline__ const uint8_t* piece_at(const DownArgs& g, int p, int piece) {
  const int q = threadIdx.x & 3;
  return reinterpret_cast<const uint8_t*>(
      g.act + (int64_t)p * g.I * kPieces + ((q >> 1) * kPieces + piece) * kFewTile + (q & 1) * 8);
}

// The pieces of the pairs list[p0 .. p0 + kDownRows), a piece of all of them
// after the other; past the n-th pair, of the last.
using DownRows = BfRows<kDownRows * kPieces / 4, 64 * kPieces>;
static_assert(kDownRows == 4, "a load of BfRows is one piece of the pairs");

__device__ __forceinline__ DownRows down_rows(const DownArgs& g, const uint16_t* list, int p0,
                                              int n) {
  DownRows rows;
  const int c = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int piece = 0; piece < kPieces; ++piece)
    rows.p[piece] = piece_at(g, list[min(p0 + c, n - 1)], piece);
  return rows;
}

// Outputs h0 .. h0 + 31 of the pairs list[p0 .. p0 + kDownRows), K split over
// the waves.
__device__ __forceinline__ void down_tile(const DownArgs& g, int64_t row, int h0,
                                          const uint16_t* list, int p0, int n, uint8_t* lds) {
  two_tiles(g.w2, g.w2_s, row, row + kFewTile, g.I / 32, down_rows(g, list, p0, n), lds);
  for (int i = threadIdx.x; i < 32 * kDownRows; i += blockDim.x) {
    const int r = i & 31, c = i >> 5;
    if (p0 + c >= n) continue;
    float sum = 0.0f;
#pragma unroll
    for (int piece = kPieces - 1; piece >= 0; --piece)
      sum += tile_sum(lds, r >> 4, r & 15, piece * kDownRows + c);
    g.part[(int64_t)list[p0 + c] * g.H + h0 + r] = sum;
  }
}

// The same with a tile a wave, over all of I.
__device__ __forceinline__ void down_wave(const DownArgs& g, int64_t row, int h0,
                                          const uint16_t* list, int p0, int n, uint8_t* lds) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  const int IB = g.I / 32;
  const uint8_t* wc[2] = {g.w2 + row * IB * 16, g.w2 + (row + kFewTile) * IB * 16};
  const uint8_t* ws[2] = {g.w2_s + row * IB, g.w2_s + (row + kFewTile) * IB};
  v4f_t acc[2] = {v4f_t{}, v4f_t{}};
  few_stream<2, true>(wc, ws, [](int, int r) { return r; }, down_rows(g, list, p0, n), IB, 0, 1,
                      lds, acc);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    // The sum of the pieces' columns.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = c < kDownRows * kPieces ? acc[t][i] : 0.0f;
      sum += __shfl_xor(sum, kDownRows);
      sum += __shfl_xor(sum, 2 * kDownRows);
      acc[t][i] = sum;
    }
    if (c < kDownRows && p0 + c < n)
      *reinterpret_cast<v4f_t*>(g.part + (int64_t)list[p0 + c] * g.H + h0 + t * kFewTile +
                                4 * (lane >> 4)) = acc[t];
  }
}

// A workgroup takes 32 outputs of an expert, or, with kWaveTiles, each of its
// waves does.
template <bool kWaveTiles>
__global__ __launch_bounds__(64 * kTileWaves) void moe_down_kernel(
    DownArgs g, const int32_t* __restrict__ ids, int pairs) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t list[kMaxPairs];
  const int e = blockIdx.y;
  const int n = list_pairs(ids, pairs, e, list);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int h0 = (kWaveTiles ? blockIdx.x * kTileWaves + wave : blockIdx.x) * 2 * kFewTile;
  if (n == 0 || h0 >= g.H) return;
  const int64_t row = (int64_t)e * g.H + h0;
  for (int p0 = blockIdx.z * kDownRows; p0 < n; p0 += gridDim.z * kDownRows) {
    if constexpr (kWaveTiles)
      down_wave(g, row, h0, list, p0, n, lds + wave * few_lds_bytes<2, DownRows>());
    else
      down_tile(g, row, h0, list, p0, n, lds);
  }
}

// The sums of a wave's tiles over the parts of K, in LDS: red[wave][group]
// [256] of share_stream's acc.
template <int kGroups>
__device__ __forceinline__ void share_put(const v4f_t (&acc)[kGroups], uint8_t* lds) {
  auto* red = reinterpret_cast<float*>(lds) + (threadIdx.x >> 6) * kGroups * 256 +
              (threadIdx.x & 63);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kGroups; ++q)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[q * 256 + v * 64] = acc[q][v];
  __syncthreads();
}

template <int kGroups>
__device__ __forceinline__ float share_get(const uint8_t* lds, int tile, int r, int c,
                                           int parts) {
  const float* p = reinterpret_cast<const float*>(lds) + (tile * kGroups + c / 16) * 256 +
                   (r & 3) * 64 + (r >> 2) * 16 + c % 16;
  float sum = p[0];
  for (int q = 1; q < parts; ++q) sum += p[q * kShareTiles * kGroups * 256];
  return sum;
}

// Many pairs an expert. A workgroup takes 64 outputs of an expert and its waves
// share the pieces of 10 pairs, or of 5, so a weight is decoded once for two
// products.
constexpr int kDensePairs = 32 / kPieces;

__global__ __launch_bounds__(64 * kShareTiles * kDenseParts) void moe_dense_down_kernel(
    DownArgs g, const int32_t* __restrict__ ids, int pairs) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint16_t list[kMaxPairs];
  const int e = blockIdx.y;
  const int n = list_pairs(ids, pairs, e, list);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int parts = (blockDim.x >> 6) / kShareTiles;
  const int tile = wave % kShareTiles, part = wave / kShareTiles;
  const int h0 = blockIdx.x * kShareTiles * kFewTile;
  const int last = min(g.H - h0, kShareTiles * kFewTile) - 1;
  const int64_t row = (int64_t)e * g.H + h0;
  const int IB = g.I / 32;
  const auto take = [&](auto xl, int p0) {
    constexpr int XL = decltype(xl)::value, kGroups = XL / 4, kRows = 4 * XL / kPieces;
    v4f_t acc[kGroups] = {};
    share_stream<XL, 64 * kPieces>(
        g.w2 + row * IB * 16, g.w2_s + row * IB,
        [&](int r) { return min(kFewTile * tile + r, last); },
        [&](int c) {
          return piece_at(g, list[min(p0 + c % kRows, n - 1)], min(c / kRows, kPieces - 1));
        },
        IB, tile, part, parts, lds, acc);
    share_put(acc, lds);
    for (int i = threadIdx.x; i < 64 * kRows; i += blockDim.x) {
      const int r = i & 63, c = i >> 6;
      if (p0 + c >= n || r > last) continue;
      float sum = 0.0f;
#pragma unroll
      for (int piece = kPieces - 1; piece >= 0; --piece)
        sum += share_get<kGroups>(lds, r >> 4, r & 15, piece * kRows + c, parts);
      g.part[(int64_t)list[p0 + c] * g.H + h0 + r] = sum;
    }
    __syncthreads();
  };
  for (int p0 = blockIdx.z * kDensePairs; p0 < n; p0 += gridDim.z * kDensePairs) {
    if (n - p0 <= 16 / kPieces)
      take(std::integral_constant<int, 4>{}, p0);
    else
      take(std::integral_constant<int, 8>{}, p0);
  }
}

// y[t] = the weighted sum of the token's parts, in order of j. The parts are
// loaded before it is known which count, eight at a time: an absent pair's
// part is memory that nothing wrote, and is not added.
constexpr int kSumThreads = 64;

template <bool kOutFp32>
__global__ __launch_bounds__(kSumThreads) void moe_sum_kernel(const float* __restrict__ part,
                                                              const int32_t* __restrict__ ids,
                                                              const float* __restrict__ weights,
                                                              int H, int E, int top_k,
                                                              void* __restrict__ y) {
  const int h = (blockIdx.x * kSumThreads + threadIdx.x) * 2;
  const int64_t t = blockIdx.y;
  if (h >= H) return;
  float s0 = 0.0f, s1 = 0.0f;
  for (int j0 = 0; j0 < top_k; j0 += 8) {
    float2 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = *reinterpret_cast<const float2*>(part + (t * top_k + min(j0 + j, top_k - 1)) * H + h);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t p = t * top_k + min(j0 + j, top_k - 1);
      const int e = ids[p];
      const float w = weights[p];
      if (j0 + j < top_k && e >= 0 && e < E) {
        s0 = fmaf(w, v[j].x, s0);
        s1 = fmaf(w, v[j].y, s1);
      }
    }
  }
  const float sum[2] = {s0, s1};  // y is 4-byte aligned and no more
  if constexpr (kOutFp32)
    __builtin_memcpy(static_cast<float*>(y) + t * H + h, &sum, 8);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(y) + t * H + h) = pack_bf16x2(s0, s1);
}

// From here on (two waves a SIMD) each wave takes a tile and all of its K;
// with fewer tiles K is split over a workgroup's waves. 32 tokens, 128 experts
// of 2048 x 768 (6144 and 8192 tiles): the call 73 us against 83; 7 tokens, 10
// experts of 1056 x 544 (340 tiles): 6.9 + 6.6 us against 5.3 + 5.3.
constexpr int64_t kManyTiles = 2048;

// Rounds of `most` pairs that an expert with a quarter more than the average
// needs.
int expected_rounds(int pairs, int E, int most) {
  return std::max(1, (5 * pairs / (4 * E) + most - 1) / most);
}

// `tiles` tiles of each expert, of `units` units of K and `columns` pairs at a
// time. Where that leaves room for them, an expert's rounds are workgroups of
// their own: up to four of those fit a CU (32 tokens, 4 experts of 2048 x
// 1536, top 4: 384 workgroups 13.5 us, 768 11.4; 16 experts of 512 x 512, top
// 8: 512 7.4 us, 1024 5.9; 8 experts of 1024 x 1440, top 8: 720 13.3 us, 1440
// 14.1).
template <class Kernel, class Args>
hipError_t launch_tiles(Kernel kernel, int columns, int lds_per_wave, const Args& g, int64_t tiles,
                        int64_t units, bool wave_tiles, const int32_t* ids, int pairs, int E,
                        hipStream_t stream) {
  const int waves = wave_tiles ? kTileWaves : even_waves((int)units, kTileWaves);
  const int64_t room = std::max<int64_t>(1, 1024 / (tiles * E));
  const int rounds = (int)std::min<int64_t>(room, expected_rounds(pairs, E, columns));
  const dim3 grid(wave_tiles ? (tiles + kTileWaves - 1) / kTileWaves : tiles, E,
                  wave_tiles ? 1 : rounds);
  hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), lds_per_wave * waves, stream, g, ids,
                     pairs);
  return hipGetLastError();
}

// Whether every pair reads its expert's weights for itself. One token's
// experts differ anyway, and several tokens seldom share one while there are
// fewer pairs than experts (128 experts of 2048 x 768, top 8: 2 tokens 12.4 us
// against 23.3 by experts, 8 tokens 31.8 against 42.1, 16 tokens 53.2 against
// 56.6, 24 tokens 73.7 against 67.1). The less the pairs read, the better the
// caches serve what they share, and the launch less counts: up to 1.5 pairs an
// expert with 256 MiB (5 x 480 x 4640, 17 experts, top 3, 53 MB, 14.9 against
// 19.6; 22 x 2848 x 288, 125 top 7, 40.6 against 56.4; 8 x 4096 x 1440, 12 top
// 2, 150 MB, 27.8 against 28.9; 4 x 4096 x 14336, 8 top 2, 749 MB, 127.6
// against 117.4), up to four with 64 MiB (31 x 352 x 576, 76 top 6, 60 MB, 15.4
// against 19.4; 14 x 1792 x 576, 16 top 4, 92 MB, 18.8 against 18.0).
bool by_pairs(int T, int H, int I, int E, int top_k) {
  const int64_t pairs = (int64_t)T * top_k, bytes = pairs * 3 * H * I / 32 * 17;
  return T == 1 || pairs < E ||
         (2 * pairs <= 3 * (int64_t)E && bytes <= (int64_t)256 << 20) ||
         (pairs <= 4 * (int64_t)E && bytes <= (int64_t)64 << 20);
}

// What a call of moe works on.
struct MoeArgs {
  const uint8_t* x;
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  const uint8_t *w13, *w13_s, *w2, *w2_s;
  int T, H, I, E, top_k;
  bool out_fp32;
  void* y;
  float* workspace;
};

hipError_t launch_pairs(const MoeArgs& m, hipStream_t stream) {
  const int HB = m.H / 32, IB = m.I / 32;
  const int columns = 2 * (HB <= 16 ? 4 : HB <= 32 ? 2 : 1) * (HB <= 64 ? kShortWaves : 1);
  const int up_waves = HB <= 64 ? kShortWaves : even_waves((HB + 63) / 64, kMaxWaves);
  hipLaunchKernelGGL(HB <= 16   ? moe_pair_up_short_kernel<16>
                     : HB <= 32 ? moe_pair_up_short_kernel<32>
                     : HB <= 64 ? moe_pair_up_short_kernel<64>
                                : moe_pair_up_kernel,
                     dim3(m.I / columns, m.T * m.top_k), dim3(64 * up_waves), 0, stream, m.x,
                     m.ldx, m.ids, m.w13, m.w13_s, HB, m.I, m.E, m.top_k, m.workspace);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int waves = even_waves((m.top_k * IB + 63) / 64, kPairDownWaves);
  hipLaunchKernelGGL(m.out_fp32 ? moe_pair_down_kernel<true> : moe_pair_down_kernel<false>,
                     dim3(m.H / kPairDownRows, m.T), dim3(64 * waves),
                     waves * LaneBlocks<8>::kBytes, stream, m.workspace, m.ids, m.weights, m.w2,
                     m.w2_s, m.H, IB, m.E, m.top_k, m.y);
  return hipGetLastError();
}

hipError_t launch_experts(const MoeArgs& m, hipStream_t stream) {
  const int pairs = m.T * m.top_k, HB = m.H / 32, IB = m.I / 32, E = m.E;
  // Workspace: the pairs' parts of y, then the activations' pieces.
  float* part = m.workspace;
  auto* act = reinterpret_cast<uint16_t*>(part + (int64_t)pairs * m.H);
  const UpArgs up = {m.x, m.ldx, m.w13, m.w13_s, act, HB, m.I, m.top_k};
  const int64_t up_tiles = m.I / kFewTile, up_units = (HB + kUnitBlocks - 1) / kUnitBlocks;
  const bool up_waves = up_tiles * E >= kManyTiles;
  const auto launch_up = [&](auto kernel, int columns, int lds) {
    return launch_tiles(kernel, columns, lds, up, up_tiles, up_units, up_waves, m.ids, pairs, E,
                        stream);
  };
  // Columns for up to 16 pairs in the first kernel cost registers, and waves,
  // where most experts have few: from 4 pairs an expert on they pay, or cost 3%
  // (the call with 8 and with 16: 64 experts of 1024 x 1024, pairs an expert 2:
  // 31.7 and 32.6 us, 4: 38.1 and 39.2, 6: 45.5 and 44.9, 16: 84.5 and 78.9;
  // 64 of 4096 x 1024, 1.6: 88.1 and 96.3; 128 of 2048 x 768, 4: 93.5 and 89.9;
  // 8 of 4096 x 14336, 4: 183 and 185, 6: 218 and 214).
  hipError_t e;
  if (pairs >= 4 * E)
    e = launch_up(up_waves ? moe_up_kernel<4, true> : moe_up_kernel<4, false>, 16,
                  few_lds_bytes<2, BfRows<4>>());
  else
    e = launch_up(up_waves ? moe_up_kernel<2, true> : moe_up_kernel<2, false>, 8,
                  few_lds_bytes<2, BfRows<2>>());
  if (e != hipSuccess) return e;
  const DownArgs down = {act, m.w2, m.w2_s, part, m.H, m.I};
  const int64_t down_tiles = m.H / (2 * kFewTile);
  const int64_t down_units = (IB + kUnitBlocks - 1) / kUnitBlocks;
  const bool down_waves = down_tiles * E >= kManyTiles;
  // Many pairs an expert and few tiles, but a workgroup a CU. The call with this
  // kernel and without: 32 tokens, 4 experts of 2048 x 1536, top 4, 25.5 and
  // 28.9 us; 64 tokens, 8 of 4096 x 14336, top 2, 333 and 383; 32 of 1024 x
  // 1024, 8 pairs each, 28.6 and 31.3; 32 tokens through all 8 of 1024 x 1440
  // 29.4 and 29.8. Fewer pairs (12 of 4096 x 1440, 4 each: 42.2 and 41.7) or
  // many tiles (128 of 2048 x 768, 8 each: 143 and 121; 64 of 1024 x 1024, 16
  // each: 84.6 and 78.8) do not pay.
  const int64_t blocks = (m.H + kShareTiles * kFewTile - 1) / (kShareTiles * kFewTile);
  const int rounds = std::min(8, expected_rounds(pairs, E, kDensePairs));
  if (pairs >= 8 * E && !down_waves && blocks * E * rounds >= 256) {
    const int parts = IB > kUnitBlocks ? kDenseParts : 1;
    const int lds = std::max(share_lds_bytes<4>(parts), share_lds_bytes<8>(parts));
    hipLaunchKernelGGL(moe_dense_down_kernel,
                       dim3(blocks, E, rounds), dim3(64 * kShareTiles * parts), lds, stream, down,
                       m.ids, pairs);
    e = hipGetLastError();
  } else {
    e = launch_tiles(down_waves ? moe_down_kernel<true> : moe_down_kernel<false>, kDownRows,
                     few_lds_bytes<2, DownRows>(), down, down_tiles, down_units, down_waves, m.ids,
                     pairs, E, stream);
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(m.out_fp32 ? moe_sum_kernel<true> : moe_sum_kernel<false>,
                     dim3((m.H / 2 + kSumThreads - 1) / kSumThreads, m.T), dim3(kSumThreads), 0,
                     stream, part, m.ids, m.weights, m.H, E, m.top_k, m.y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(const void* x, int64_t ldx, const int32_t* ids, const float* weights,
                      const void* w13, const void* w13_s, const void* w2, const void* w2_s, int T,
                      int H, int I, int E, int top_k, bool out_fp32, void* y, void* workspace,
                      hipStream_t stream) {
  const MoeArgs m = {static_cast<const uint8_t*>(x),    ldx,
                     ids,                               weights,
                     static_cast<const uint8_t*>(w13),  static_cast<const uint8_t*>(w13_s),
                     static_cast<const uint8_t*>(w2),   static_cast<const uint8_t*>(w2_s),
                     T, H, I, E, top_k, out_fp32, y, static_cast<float*>(workspace)};
  return by_pairs(T, H, I, E, top_k) ? launch_pairs(m, stream) : launch_experts(m, stream);
}

}  // namespace mxfp4
