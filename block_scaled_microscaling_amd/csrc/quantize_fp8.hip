// BF16 -> FP8 quantize for gfx950 with a scale for each block of 128: E4M3 or
// E5M2 codes, the scale the smallest power of two that brings the block's
// largest finite magnitude within the type (fp8.h). Blocks are 1 x 128 (an
// activation) or 128 x 128 (a weight); either form can be written together
// with that of X^T in one pass over X, which the weight gradient's and the
// input gradient's products contract over.
//
// All of them are bound by memory: 2 bytes read and 1 + 1/128 written per
// element and form (8192 x 8192 both ways 50.7 us, 5.3 TB/s; 28672 x 4096 in
// 128 x 128 blocks both ways 93 us, 5.1 TB/s, a large copy's rate; 1 x 4096
// 2 us beside a launch).
//
// Rows alone (quantize_fp8_rows_kernel): 16 lanes hold one block, 16 bytes (8
// values) each, so a wave reads 4 blocks, 1 KiB, and its codes leave as whole
// 128-byte lines; the maximum is taken on the bits (packed 16-bit integers)
// and finished over the 16 lanes with four DPP moves.
//
// Tiles (quantize_fp8_tile_kernel): a workgroup of 256 threads holds a 128 x
// 128 tile, thread (g, c) rows 8 g .. 8 g + 7 of columns 8 c .. 8 c + 7, so a
// row's block is 16 lanes as above, and a column's block is the 16 groups g:
// two shuffles within a wave and one exchange of 256 bytes a wave through
// LDS. A thread's 8 x 8 patch is turned in registers (byte permutes pair two
// rows of one column for the conversion) and the transposed codes go through
// LDS, so that they too leave as whole 128-byte lines.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kFp8Block;
constexpr int kMaxGrid = 1 << 20;  // workgroups; the kernels stride over the rest

__device__ __forceinline__ int pair_max(i16x2_t m) { return max((int)m.x, (int)m.y); }

// Blocks go in flat order over [M, ceil(K / 128)]; kFlat: rows are whole
// blocks and lie one behind the other, so that the order is that of memory.
template <Fp8Type kType, bool kFlat>
__global__ __launch_bounds__(kThreads) void quantize_fp8_rows_kernel(Fp8QuantArgs p, int64_t blocks,
                                                                     int kblocks) {
  constexpr int kPer = 4;  // blocks of 16 lanes in flight
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  constexpr int kGroups = kThreads / 16;
  for (int64_t b0 = (int64_t)blockIdx.x * (kGroups * kPer); b0 < blocks;
       b0 += (int64_t)gridDim.x * (kGroups * kPer)) {
    u32x4_t v[kPer];
    int64_t out[kPer];
    bool in[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t b = b0 + i * kGroups + g;
      int64_t at = b * kTile + 8 * c;
      in[i] = b < blocks;
      out[i] = at;
      if constexpr (!kFlat) {
        const int64_t row = b / kblocks;
        const int col = (int)(b - row * kblocks) * kTile + 8 * c;
        in[i] = in[i] && col < p.K;
        at = row * p.ldx + col;
        out[i] = row * p.K + col;
      }
      v[i] = u32x4_t{};
      if (in[i]) v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p.x + at));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t b = b0 + i * kGroups + g;
      const uint32_t byte = fp8_row_scale<kType>(v[i]);
      const uint2 code = fp8_encode_chunk<kType>(v[i], fp8_scale_value(byte));
      if (in[i]) *reinterpret_cast<uint2*>(p.codes + out[i]) = code;
      if (c == 0 && b < blocks) store_scale(p.scales, b, byte, p.scale_f32);
    }
  }
}

template <Fp8Type kType, bool kSquare, bool kBoth>
__global__ __launch_bounds__(kThreads) void quantize_fp8_tile_kernel(Fp8QuantArgs p, int mblocks,
                                                                     int kblocks) {
  __shared__ __align__(16) uint8_t turned[kBoth ? kTile * kTile : 16];
  __shared__ __align__(16) i16x2_t tops[4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = tid & 15, g = tid >> 4;
  const int64_t Mp = ((int64_t)p.M + 15) / 16 * 16;
  const int64_t tiles = (int64_t)mblocks * kblocks;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int mb = (int)(t / kblocks), kb = (int)(t - (int64_t)mb * kblocks);
    const int64_t m0 = (int64_t)mb * kTile + 8 * g;
    const int k0 = kb * kTile + 8 * c;
    u32x4_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = u32x4_t{};
      if (m0 + i < p.M && k0 < p.K)
        v[i] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(p.x + (m0 + i) * p.ldx + k0));
    }
    // Columns' maxima of the wave's 32 rows, columns 8 c + 2 j, + 1 in m[j].
    i16x2_t m[4];
    if constexpr (kBoth || kSquare) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        i16x2_t a = {(short)kAmaxBias, (short)kAmaxBias};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = v[i][j];
          a = max_pair(a, biased_abs_pair(w));
        }
        int o = __shfl_xor(__builtin_bit_cast(int, a), 16);
        a = max_pair(a, __builtin_bit_cast(i16x2_t, o));
        o = __shfl_xor(__builtin_bit_cast(int, a), 32);
        m[j] = max_pair(a, __builtin_bit_cast(i16x2_t, o));
      }
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) tops[wave][4 * c + j] = m[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m[j] = max_pair(max_pair(tops[0][4 * c + j], tops[1][4 * c + j]),
                        max_pair(tops[2][4 * c + j], tops[3][4 * c + j]));
    }
    uint32_t square = 0;
    if constexpr (kSquare) {
      const int top = row16_max(pair_max(max_pair(max_pair(m[0], m[1]), max_pair(m[2], m[3]))));
      square = fp8_scale_byte_bf16<kType>((uint32_t)(top - kAmaxBias));
      if (tid == 0) {
        store_scale(p.scales, (int64_t)mb * kblocks + kb, square, p.scale_f32);
        if (kBoth) store_scale(p.scales_t, (int64_t)kb * mblocks + mb, square, p.scale_f32);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t byte = square;
      if constexpr (!kSquare) {
        byte = fp8_row_scale<kType>(v[i]);
        if (c == 0 && m0 + i < p.M)
          store_scale(p.scales, (m0 + i) * kblocks + kb, byte, p.scale_f32);
      }
      const uint2 code = fp8_encode_chunk<kType>(v[i], fp8_scale_value(byte));
      if (m0 + i < p.M && k0 < p.K)
        *reinterpret_cast<uint2*>(p.codes + (m0 + i) * p.K + k0) = code;
    }
    if constexpr (kBoth) {
      // Column 8 c + j's 8 bytes of group g at slot g ^ c of its 128-byte
      // row: the lanes of one store fall on all slots equally.
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t byte = square;
        if constexpr (!kSquare) {
          byte = fp8_scale_byte_bf16<kType>((uint32_t)((int)(j & 1 ? m[j / 2].y : m[j / 2].x) -
                                                       kAmaxBias));
          if (g == 0 && k0 + j < p.K)
            store_scale(p.scales_t, (int64_t)(k0 + j) * mblocks + mb, byte, p.scale_f32);
        }
        const float scale = fp8_scale_value(byte);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = v[2 * i][j / 2], hi = v[2 * i + 1][j / 2];
          w[i] = __builtin_amdgcn_perm(hi, lo, j & 1 ? 0x07060302u : 0x05040100u);
        }
        uint2 code;
        code.x = fp8_pair_bf16<kType, true>(fp8_pair_bf16<kType, false>(0, w[0], scale), w[1],
                                            scale);
        code.y = fp8_pair_bf16<kType, true>(fp8_pair_bf16<kType, false>(0, w[2], scale), w[3],
                                            scale);
        *reinterpret_cast<uint2*>(turned + (8 * c + j) * kTile + 8 * (g ^ c)) = code;
      }
      __syncthreads();
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int col = 32 * it + (tid >> 3), q = tid & 7, cc = col >> 3;
        uint4 w = *reinterpret_cast<const uint4*>(turned + col * kTile + 8 * ((2 * q) ^ (cc & 14)));
        if (cc & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        const int64_t mm = (int64_t)mb * kTile + 16 * q;
        if (mm < Mp && kb * kTile + col < p.K)
          *reinterpret_cast<uint4*>(p.codes_t + (int64_t)(kb * kTile + col) * Mp + mm) = w;
      }
    }
    __syncthreads();
  }
}

template <Fp8Type kType>
hipError_t launch(const Fp8QuantArgs& a, int block_rows, hipStream_t stream) {
  const int kblocks = (int)(((int64_t)a.K + kTile - 1) / kTile);
  const int mblocks = (int)(((int64_t)a.M + kTile - 1) / kTile);
  const dim3 threads(kThreads);
  if (block_rows == 1 && !a.codes_t) {
    const int64_t blocks = (int64_t)a.M * kblocks;
    const int64_t wgs = (blocks + 63) / 64;
    const dim3 grid((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid));
    if (a.K % kTile == 0 && (a.M == 1 || a.ldx == a.K))
      hipLaunchKernelGGL((quantize_fp8_rows_kernel<kType, true>), grid, threads, 0, stream, a,
                         blocks, kblocks);
    else
      hipLaunchKernelGGL((quantize_fp8_rows_kernel<kType, false>), grid, threads, 0, stream, a,
                         blocks, kblocks);
    return hipGetLastError();
  }
  const int64_t tiles = (int64_t)mblocks * kblocks;
  const dim3 grid((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid));
  if (block_rows == 1)
    hipLaunchKernelGGL((quantize_fp8_tile_kernel<kType, false, true>), grid, threads, 0, stream, a,
                       mblocks, kblocks);
  else if (a.codes_t)
    hipLaunchKernelGGL((quantize_fp8_tile_kernel<kType, true, true>), grid, threads, 0, stream, a,
                       mblocks, kblocks);
  else
    hipLaunchKernelGGL((quantize_fp8_tile_kernel<kType, true, false>), grid, threads, 0, stream, a,
                       mblocks, kblocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const Fp8QuantArgs& a, int block_rows, Fp8Type type,
                               hipStream_t stream) {
  return type == kE4M3 ? launch<kE4M3>(a, block_rows, stream)
                       : launch<kE5M2>(a, block_rows, stream);
}

}  // namespace mxfp4
