// The backward pass of act = silu(g) u between the gated MLP's two products,
// with the quantize that both of its products need: from dact [M, I] and the
// g, u [M, 2 I] kept by the forward product (all BF16),
//   du = dact g s,   dg = dact u s (1 + g (1 - s)),   s = 1 / (1 + exp(-g)),
// in FP32, and [dg, du] quantized straight from FP32 in 1 x 128 blocks along
// its rows (the operand of dx = dgu W13) and along its columns (the rows of
// dgu^T, the operand of dW13 = dgu^T x). Neither gradient is written in BF16.
//
// Bound by memory: 6 bytes read and 2 (1 + 1/128) x 2 written per element of
// act; the VALU's share is near it, so magnitudes are compared as floats, two in
// one v_max3. One workgroup of 1024 threads holds a 128 x 128 tile of act, thread
// (g, c) rows 4 g .. + 3 of columns 4 c .. + 3 of both gradients in registers (32
// values, four waves a SIMD: 16384 x 14336 608 us, 3.9 TB/s; with 64 values in 512
// threads it was two waves, 667 us; with eight waves, whose registers spill, 597,
// but 4096 x 4096 50 instead of 45). A row's block is 32 lanes (DPP moves and one swap
// of lanes), a column's the 32 groups g: one swap, which also puts two columns
// into one register, then a maximum in LDS. The transposed codes go through LDS,
// so that all codes leave as whole 128-byte lines.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kTile = kFp8Block;
constexpr int kPatch = 4;          // rows and columns of a thread
constexpr int kMaxGrid = 1 << 20;  // workgroups; the kernel strides over the rest

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint2 load_once(const uint16_t* x) {
  typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
  const u32x2_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(x));
  return make_uint2(v[0], v[1]);
}

// |v|; 0 for infinities and NaN where kFinite (a maximum passes over NaN).
template <bool kFinite>
__device__ __forceinline__ float magnitude(float v) {
  const float m = __builtin_fabsf(v);
  return kFinite && !(m < __builtin_inff()) ? 0.0f : m;
}

// Maxima of two values over pairs of half waves: a's in the lower half, b's in
// the upper one.
__device__ __forceinline__ float merge32_max(float a, float b) {
  const auto s =
      __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
// Maximum over the 32 lanes of a half wave.
__device__ __forceinline__ float half_max(float v) {
  const uint32_t m = (uint32_t)row16_max((int)__float_as_uint(v));  // not negative: orders as int
  const auto s = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

template <Fp8Type kType>
__global__ __launch_bounds__(kThreads, 4) void swiglu_fp8_backward_kernel(SwigluBackwardArgs p,
                                                                          int mblocks,
                                                                          int iblocks) {
  __shared__ __align__(16) uint8_t turned[2][kTile * kTile];
  __shared__ __align__(16) int tops[2][kTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = tid & 31, g = tid >> 5;
  const int64_t Mp = ((int64_t)p.M + 15) / 16 * 16;
  const int64_t tiles = (int64_t)mblocks * iblocks;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int mb = (int)(t / iblocks), ib = (int)(t - (int64_t)mb * iblocks);
    const int64_t m0 = (int64_t)mb * kTile + kPatch * g;
    const int i0 = ib * kTile + kPatch * c;
    if (tid < 2 * kTile) (&tops[0][0])[tid] = 0;

    uint2 vd[kPatch], vg[kPatch], vu[kPatch];
#pragma unroll
    for (int i = 0; i < kPatch; ++i) {
      vd[i] = vg[i] = vu[i] = make_uint2(0, 0);
      if (m0 + i < p.M) {
        const uint16_t* gu = p.gu + (m0 + i) * 2 * p.I + i0;
        vd[i] = load_once(p.dact + (m0 + i) * p.I + i0);
        vg[i] = load_once(gu);
        vu[i] = load_once(gu + p.I);
      }
    }
    float d[2][kPatch][kPatch];  // dg, du
    float most = 0;
#pragma unroll
    for (int i = 0; i < kPatch; ++i)
#pragma unroll
      for (int j = 0; j < kPatch; ++j) {
        const uint32_t wd = j < 2 ? vd[i].x : vd[i].y, wg = j < 2 ? vg[i].x : vg[i].y;
        const uint32_t wu = j < 2 ? vu[i].x : vu[i].y;
        const float dy = j & 1 ? bf16_hi(wd) : bf16_lo(wd);
        const float gg = j & 1 ? bf16_hi(wg) : bf16_lo(wg);
        const float uu = j & 1 ? bf16_hi(wu) : bf16_lo(wu);
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-gg));
        const float ds = dy * s;
        d[0][i][j] = ds * uu * fmaf(gg, 1.0f - s, 1.0f);
        d[1][i][j] = ds * gg;
        most = __builtin_fmaxf(__builtin_fmaxf(most, __builtin_fabsf(d[0][i][j])),
                               __builtin_fabsf(d[1][i][j]));
      }
    float row_top[2][kPatch];
    const auto find_tops = [&](auto finite) {
      constexpr bool kFinite = decltype(finite)::value;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int j = 0; j < kPatch; j += 2) {
          float col[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < kPatch; ++i)
              col[e] = __builtin_fmaxf(col[e], magnitude<kFinite>(d[w][i][j + e]));
          atomicMax(&tops[w][kPatch * c + j + (lane >> 5)],
                    (int)__float_as_uint(merge32_max(col[0], col[1])));
        }
#pragma unroll
        for (int i = 0; i < kPatch; ++i) {
          float row = 0;
#pragma unroll
          for (int j = 0; j < kPatch; ++j)
            row = __builtin_fmaxf(row, magnitude<kFinite>(d[w][i][j]));
          row_top[w][i] = half_max(row);
        }
      }
    };
    // tops is clear, and the last tile's turned has been read. Infinities are
    // rare, so leaving them out of the maxima is a path of its own.
    if (__syncthreads_or(!(most < __builtin_inff())))
      find_tops(std::true_type());
    else
      find_tops(std::false_type());
    // Rows.
    const int64_t kblocks = 2 * (int64_t)iblocks;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < kPatch; ++i) {
        const uint32_t byte = fp8_scale_byte_f32<kType>(__float_as_uint(row_top[w][i]));
        const float s = fp8_scale_value(byte);
        const float* v = d[w][i];
        const uint32_t code =
            fp8_pair_f32<kType, true>(fp8_pair_f32<kType, false>(0, v[0], v[1], s), v[2], v[3], s);
        if (m0 + i < p.M) {
          *reinterpret_cast<uint32_t*>(p.codes + (m0 + i) * 2 * p.I + (int64_t)w * p.I + i0) =
              code;
          if (c == 0) p.scales[(m0 + i) * kblocks + w * iblocks + ib] = (uint8_t)byte;
        }
      }
    __syncthreads();  // tops is whole
    // Columns: column 4 c + j's 4 bytes of group g at dword g ^ c of its 128-byte
    // row, so that the lanes of one store fall on all banks.
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int j = 0; j < kPatch; ++j) {
        const uint32_t byte = fp8_scale_byte_f32<kType>((uint32_t)tops[w][kPatch * c + j]);
        const float s = fp8_scale_value(byte);
        *reinterpret_cast<uint32_t*>(turned[w] + (kPatch * c + j) * kTile + 4 * (g ^ c)) =
            fp8_pair_f32<kType, true>(fp8_pair_f32<kType, false>(0, d[w][0][j], d[w][1][j], s),
                                      d[w][2][j], d[w][3][j], s);
        if (g == 0) p.scales_t[((int64_t)w * p.I + i0 + j) * mblocks + mb] = (uint8_t)byte;
      }
    __syncthreads();  // turned is whole
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int col = tid >> 3, q = tid & 7, x = col / kPatch;
      uint4 v = *reinterpret_cast<const uint4*>(turned[w] + col * kTile + 16 * (q ^ (x >> 2)));
      if (x & 1) v = make_uint4(v.y, v.x, v.w, v.z);
      if (x & 2) v = make_uint4(v.z, v.w, v.x, v.y);
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
