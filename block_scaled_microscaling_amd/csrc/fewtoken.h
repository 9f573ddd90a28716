// Shared by the few-token kernels (gemv.hip, moe.hip): the product of 16
// MXFP4 weight rows with up to 16 BF16 activation rows on
// v_mfma_f32_16x16x32_bf16, and the launchers that api_fewtoken.hip calls.
//
// Operands. The weight rows are the MFMA's first operand and the activation
// rows ("tokens") its second: lane l holds 8 consecutive k of weight row
// l % 16 and of token l % 16, both for the K group l / 16, and accumulator
// register v of lane l is output (row 4 (l / 16) + v, token l % 16). The
// sum over k does not care which k the four groups stand for, so group g
// takes whole 32-element blocks: one 16-byte load is the codes of one block
// of the lane's row, and its 8-element quarters feed four MFMAs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gfx950.h"

namespace mxfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

constexpr int kFewTile = 16;        // weight rows and tokens of one MFMA
constexpr int kFewChunkBlocks = 8;  // 32-element blocks a wave takes per step (256 k)

// Eight E2M1 codes (element 2i in bits 3:0 of byte i) times 2^(byte - 127),
// in BF16, exact; scale carries the UE8M0 byte in its float exponent field.
__device__ __forceinline__ bf16x8_t decode8(uint32_t w, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return (bf16x8_t){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float scale_of_byte(uint32_t byte) {
  return __uint_as_float(byte << 23);
}

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

// Launchers: arguments are validated by the caller.
hipError_t launch_gemv(const void* x, int64_t ldx, const void* codes, const void* scales, int M,
                       int N, int K, bool out_fp32, void* y, hipStream_t stream);
hipError_t launch_moe_route(const void* x, int64_t ldx, const void* router, int T, int H, int E,
                            int top_k, bool renormalize, int32_t* ids, float* weights,
                            double* logits, hipStream_t stream);
hipError_t launch_moe(const void* x, int64_t ldx, const int32_t* ids, const float* weights,
                      const void* w13, const void* w13_s, const void* w2, const void* w2_s, int T,
                      int H, int I, int E, int top_k, bool out_fp32, void* y, uint16_t* act,
                      hipStream_t stream);

}  // namespace mxfp4
