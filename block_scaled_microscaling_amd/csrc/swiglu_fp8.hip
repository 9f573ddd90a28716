// The backward pass of act = silu(g) u between the gated MLP's two products,
// with the quantize that both of its products need: from dact [M, I] and the
// g, u [M, 2 I] kept by the forward product (all BF16),
//   du = dact g s,   dg = dact u s (1 + g (1 - s)),   s = 1 / (1 + exp(-g)),
// in FP32, and [dg, du] quantized straight from FP32 in 1 x 128 blocks along
// its rows (the operand of dx = dgu W13) and along its columns (the rows of
// dgu^T, the operand of dW13 = dgu^T x). Neither gradient is written in BF16.
//
// Bound by memory: 6 bytes read and 2 (1 + 1/128) x 2 written per element of
// act. One workgroup of 512 threads holds a 128 x 128 tile of act, thread
// (g, c) rows 4 g .. + 3 of columns 8 c .. + 7 of both gradients in registers
// (64 values), so a row's block is 16 lanes (four DPP moves) and a column's
// the 32 groups g: two shuffles, then a maximum in LDS. The transposed codes
// go through LDS, so that all codes leave as whole 128-byte lines.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = kFp8Block;
constexpr int kRows = 4;           // of a thread
constexpr int kMaxGrid = 1 << 20;  // workgroups; the kernel strides over the rest

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// |v| as an integer that orders like it; 0 for infinities and NaN.
__device__ __forceinline__ int finite_abs(float v) {
  const int b = (int)(__float_as_uint(v) & 0x7FFFFFFFu);
  return b < 0x7F800000 ? b : 0;
}

template <Fp8Type kType>
__global__ __launch_bounds__(kThreads) void swiglu_fp8_backward_kernel(SwigluBackwardArgs p,
                                                                       int mblocks, int iblocks) {
  __shared__ __align__(16) uint8_t turned[2][kTile * kTile];
  __shared__ __align__(16) int tops[2][kTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = tid & 15, g = tid >> 4;
  const int64_t Mp = ((int64_t)p.M + 15) / 16 * 16;
  const int64_t tiles = (int64_t)mblocks * iblocks;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int mb = (int)(t / iblocks), ib = (int)(t - (int64_t)mb * iblocks);
    const int64_t m0 = (int64_t)mb * kTile + kRows * g;
    const int i0 = ib * kTile + 8 * c;
    if (tid < 2 * kTile) (&tops[0][0])[tid] = 0;

    u32x4_t vd[kRows], vg[kRows], vu[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      vd[i] = vg[i] = vu[i] = u32x4_t{};
      if (m0 + i < p.M) {
        const uint16_t* gu = p.gu + (m0 + i) * 2 * p.I + i0;
        vd[i] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t*>(p.dact + (m0 + i) * p.I + i0));
        vg[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(gu));
        vu[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(gu + p.I));
      }
    }
    float d[2][kRows][8];  // dg, du
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t wd = vd[i][j / 2], wg = vg[i][j / 2], wu = vu[i][j / 2];
        const float dy = j & 1 ? bf16_hi(wd) : bf16_lo(wd);
        const float gg = j & 1 ? bf16_hi(wg) : bf16_lo(wg);
        const float uu = j & 1 ? bf16_hi(wu) : bf16_lo(wu);
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-gg));
        const float ds = dy * s;
        d[0][i][j] = ds * uu * fmaf(gg, 1.0f - s, 1.0f);
        d[1][i][j] = ds * gg;
      }
    __syncthreads();  // tops is clear, and the last tile's turned has been read
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        int top = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) top = max(top, finite_abs(d[w][i][j]));
        top = max(top, __shfl_xor(top, 16));
        top = max(top, __shfl_xor(top, 32));
        if (lane < 16) atomicMax(&tops[w][8 * c + j], top);
      }
    // Rows.
    const int64_t kblocks = 2 * (int64_t)iblocks;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        int top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, finite_abs(d[w][i][j]));
        const uint32_t byte = fp8_scale_byte_f32<kType>((uint32_t)row16_max(top));
        const float s = fp8_scale_value(byte);
        const float* v = d[w][i];
        uint2 code;
        code.x = fp8_pair_f32<kType, true>(fp8_pair_f32<kType, false>(0, v[0], v[1], s), v[2],
                                           v[3], s);
        code.y = fp8_pair_f32<kType, true>(fp8_pair_f32<kType, false>(0, v[4], v[5], s), v[6],
                                           v[7], s);
        if (m0 + i < p.M) {
          *reinterpret_cast<uint2*>(p.codes + (m0 + i) * 2 * p.I + (int64_t)w * p.I + i0) = code;
          if (c == 0) p.scales[(m0 + i) * kblocks + w * iblocks + ib] = (uint8_t)byte;
        }
      }
    __syncthreads();  // tops is whole
    // Columns: column 8 c + j's 4 bytes of group g at dword g ^ 4 (c % 8) of
    // its 128-byte row, so that the lanes of one store fall on all banks.
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t byte = fp8_scale_byte_f32<kType>((uint32_t)tops[w][8 * c + j]);
        const float s = fp8_scale_value(byte);
        const uint32_t code = fp8_pair_f32<kType, true>(
            fp8_pair_f32<kType, false>(0, d[w][0][j], d[w][1][j], s), d[w][2][j], d[w][3][j], s);
        *reinterpret_cast<uint32_t*>(turned[w] + (8 * c + j) * kTile + 4 * (g ^ (4 * (c & 7)))) =
            code;
        if (g == 0)
          p.scales_t[((int64_t)w * p.I + i0 + j) * mblocks + mb] = (uint8_t)byte;
      }
    __syncthreads();  // turned is whole
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int w = it >> 1, col = 64 * (it & 1) + (tid >> 3), q = tid & 7;
      const uint4 v =
          *reinterpret_cast<const uint4*>(turned[w] + col * kTile + 16 * (q ^ ((col >> 3) & 7)));
      const int64_t mm = (int64_t)mb * kTile + 16 * q;
      if (mm < Mp)
        *reinterpret_cast<uint4*>(p.codes_t + ((int64_t)w * p.I + ib * kTile + col) * Mp + mm) = v;
    }
  }
}

}  // namespace

hipError_t launch_swiglu_fp8_backward(const SwigluBackwardArgs& a, Fp8Type type,
                                      hipStream_t stream) {
  const int mblocks = (int)(((int64_t)a.M + kTile - 1) / kTile), iblocks = a.I / kTile;
  const int64_t tiles = (int64_t)mblocks * iblocks;
  const dim3 grid((unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid));
  if (type == kE4M3)
    hipLaunchKernelGGL((swiglu_fp8_backward_kernel<kE4M3>), grid, dim3(kThreads), 0, stream, a,
                       mblocks, iblocks);
  else
    hipLaunchKernelGGL((swiglu_fp8_backward_kernel<kE5M2>), grid, dim3(kThreads), 0, stream, a,
                       mblocks, iblocks);
  return hipGetLastError();
}

}  // namespace mxfp4
