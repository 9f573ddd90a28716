// Shared by the FP8 kernels (quantize_fp8.hip, gemm_fp8.hip, gemm_fp8_small.hip,
// gemm_fp8_tile.hip, swiglu_fp8.hip): the scale rule, conversions, the
// matrix instructions and the launchers that api_fp8.hip calls.
//
// An FP8 operand is E4M3 or E5M2 codes with one scale per block of 128
// elements of a row, or per 128 x 128 block. A scale is a power of two, held
// as its UE8M0 byte or as FP32 (a GEMM takes any FP32 scales).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gfx950.h"

namespace mxfp4 {

constexpr int kFp8Block = 128;  // elements of a row, and rows of a block, under one scale

typedef short i16x2_t __attribute__((ext_vector_type(2)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

enum Fp8Type { kE4M3 = 0, kE5M2 = 1 };

// ------------------------------------------------------------- scale rule
// The scale of a block is 2^e, e the smallest integer with amax <= T 2^e,
// T = 448 = 1.75 2^8 (E4M3) or 57344 = 1.75 2^15 (E5M2), clamped to
// [-126, 127] (UE8M0 bytes 1 .. 254, normal FP32 values). amax = f 2^E, 1 <=
// f < 2, so e = E - 8 (or - 15), plus one where f > 1.75; on the bits of a
// float with b mantissa bits, adding 2^(b - 2) - 1 carries into the exponent
// exactly where f > 1.75. Infinities and NaN do not enter amax.
template <Fp8Type kType>
constexpr int kTopExponent = kType == kE4M3 ? 8 : 15;

template <Fp8Type kType>
__device__ __forceinline__ uint32_t fp8_scale_byte_bf16(uint32_t amax_bits) {
  return (uint32_t)max((int)((amax_bits + 31) >> 7) - kTopExponent<kType>, 1);
}
template <Fp8Type kType>
__device__ __forceinline__ uint32_t fp8_scale_byte_f32(uint32_t amax_bits) {
  return (uint32_t)max((int)((amax_bits + 0x1FFFFFu) >> 23) - kTopExponent<kType>, 1);
}
__device__ __forceinline__ float fp8_scale_value(uint32_t byte) {
  return __uint_as_float(byte << 23);
}

// |x| of two BF16 values biased by 128 as signed 16-bit integers: finite ones
// order as integers and are at least 128, infinities and NaN wrap to negative
// values, so a signed maximum that starts at 128 leaves them out.
constexpr int kAmaxBias = 128;
__device__ __forceinline__ i16x2_t biased_abs_pair(uint32_t w) {
  const u16x2_t bias = {(unsigned short)kAmaxBias, (unsigned short)kAmaxBias};
  return __builtin_bit_cast(i16x2_t, (u16x2_t)(abs_pair(w) + bias));
}
__device__ __forceinline__ i16x2_t max_pair(i16x2_t a, i16x2_t b) {
  return __builtin_elementwise_max(a, b);
}

// Maximum over the 16 lanes of a DPP row (16 i .. 16 i + 15).
__device__ __forceinline__ int row16_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  return max(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false));  // row_mirror
}

// ------------------------------------------------------------ conversions
// Two values divided by the scale (exact: a power of two) and rounded to
// nearest even, into the low or the high half of `old`. Finite values are
// within the type by the scale rule; an infinity gives NaN (E4M3) or
// infinity (E5M2), NaN gives NaN.
template <Fp8Type kType, bool kHigh>
__device__ __forceinline__ uint32_t fp8_pair_bf16(uint32_t old, uint32_t w, float scale) {
  const i16x2_t o = __builtin_bit_cast(i16x2_t, old);
  if constexpr (kType == kE4M3)
    return __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, as_bf16x2(w), scale, kHigh));
  else
    return __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(o, as_bf16x2(w), scale, kHigh));
}
template <Fp8Type kType, bool kHigh>
__device__ __forceinline__ uint32_t fp8_pair_f32(uint32_t old, float a, float b, float scale) {
  const i16x2_t o = __builtin_bit_cast(i16x2_t, old);
  if constexpr (kType == kE4M3)
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, kHigh));
  else
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(o, a, b, scale, kHigh));
}

// A lane's 16 bytes (8 BF16 values): their largest finite magnitude, biased;
// the scale byte of a row's block held by 16 lanes; and their codes.
__device__ __forceinline__ i16x2_t biased_chunk_max(u32x4_t v) {
  const uint32_t a = v[0], b = v[1], c = v[2], d = v[3];
  return max_pair(max_pair(biased_abs_pair(a), biased_abs_pair(b)),
                  max_pair(biased_abs_pair(c), biased_abs_pair(d)));
}
template <Fp8Type kType>
__device__ __forceinline__ uint32_t fp8_row_scale(u32x4_t v) {
  const i16x2_t m = biased_chunk_max(v);
  const int top = row16_max(max(max((int)m.x, (int)m.y), kAmaxBias));
  return fp8_scale_byte_bf16<kType>((uint32_t)(top - kAmaxBias));
}
template <Fp8Type kType>
__device__ __forceinline__ uint2 fp8_encode_chunk(u32x4_t v, float scale) {
  const uint32_t a = v[0], b = v[1], c = v[2], d = v[3];
  uint2 r;
  r.x = fp8_pair_bf16<kType, true>(fp8_pair_bf16<kType, false>(0, a, scale), b, scale);
  r.y = fp8_pair_bf16<kType, true>(fp8_pair_bf16<kType, false>(0, c, scale), d, scale);
  return r;
}

// Scales as a kernel writes them: UE8M0 bytes or FP32.
__device__ __forceinline__ void store_scale(void* scales, int64_t at, uint32_t byte, bool f32) {
  if (f32)
    static_cast<float*>(scales)[at] = fp8_scale_value(byte);
  else
    static_cast<uint8_t*>(scales)[at] = (uint8_t)byte;
}

// ---------------------------------------------------- matrix instructions
// Two ways to multiply. The FP8 matrix instructions (f8f6f4) run at twice
// BF16's rate, with UE8M0 scales for free, but add products that lie next to
// each other in K at 14 bits below the largest of them (measured: a product
// of 2^-14 of its neighbour's is lost; random operands are off by 1.3e-5 of
// the result's rms whatever K is). That is a hundredth of a BF16 result's
// rounding, so BF16 results of many rows take it. FP32 results, and products
// bound by memory, convert the codes to BF16 (exact) and use the BF16
// instructions, which add products in FP32 (1.3e-7 at K = 8192).

// Codes 4 i .. 4 i + 3 of w as BF16 pairs, times the scale (a power of two).
template <Fp8Type kType>
__device__ __forceinline__ bf16x2_t fp8_to_bf16(uint32_t w, float scale, bool high) {
  if constexpr (kType == kE4M3)
    return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true)
                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
  else
    return high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true)
                : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false);
}
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
template <Fp8Type kType>
__device__ __forceinline__ bf16x8_t fp8x8_to_bf16(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2_t a = fp8_to_bf16<kType>(lo, scale, false), b = fp8_to_bf16<kType>(lo, scale, true);
  const bf16x2_t c = fp8_to_bf16<kType>(hi, scale, false), d = fp8_to_bf16<kType>(hi, scale, true);
  return (bf16x8_t){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float silu_f32(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// -------------------------------------------------------------- launchers
// A grid of `total` workgroups, stacked along y where x would pass 2^32 threads;
// workgroup_id() is -1 in those past the end.
inline dim3 grid_of(int64_t total, int threads) {
  const int64_t most = ((int64_t(1) << 32) - 1) / threads / 8 * 8;  // whole rounds of XCDs
  const int64_t rows = (total + most - 1) / most;
  return dim3((unsigned)(rows > 1 ? most : total), (unsigned)rows);
}
__device__ __forceinline__ int workgroup_id(int total) {
  const int64_t id = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
  return id < total ? (int)id : -1;
}

struct Fp8QuantArgs {
  const uint16_t* x;  // BF16 [M, K], rows ldx elements apart
  int64_t ldx;
  int M, K;
  uint8_t* codes;   // [M, K]
  void* scales;
  uint8_t* codes_t;  // [K, Mp], Mp = M rounded up to 16; null: rows only
  void* scales_t;
  bool scale_f32;
};
hipError_t launch_quantize_fp8(const Fp8QuantArgs& a, int block_rows, Fp8Type type,
                               hipStream_t stream);

// Tile p in the order of the workgroups: XCD x (every 8th workgroup) takes a
// contiguous run of tiles, `group` tile rows at a time, so that the tiles that
// run together on one XCD share rows of A and B in its L2.
__device__ __forceinline__ void xcd_tile(int p, int tiles_m, int tiles_n, int group, int& tm,
                                         int& tn) {
  constexpr int kXcds = 8;
  const int total = tiles_m * tiles_n;
  const int each = total / kXcds, rem = total % kXcds;
  const int xcd = p % kXcds;
  const int at = xcd * each + min(xcd, rem) + p / kXcds;
  const int width = group * tiles_n;
  const int first = at / width * group, size = min(tiles_m - first, group);
  const int in = at % width;
  tm = first + in % size;
  tn = in / size;
}

// Four UE8M0 bytes of scales from byte `at` of an array of at least four, the
// first in the low byte; those past its end are of no meaning.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* scales, int64_t at, int64_t total) {
  const int64_t p = min(at, total - 4);
  uint32_t w;
  __builtin_memcpy(&w, scales + p, 4);
  return w >> (8 * (int)(at - p) & 31);
}
// The same of an array of any length.
__device__ __forceinline__ uint32_t short_scale_word(const uint8_t* scales, int64_t at,
                                                     int64_t total) {
  if (total >= 4) return scale_word(scales, at, total);
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i)
    if (at + i < total) w |= (uint32_t)scales[at + i] << (8 * i);
  return w;
}

// Where a DMA of chunks past K reads from.
static __device__ __align__(16) const uint8_t kFp8Zeros[16] = {};

// A GEMM's operands: A [M, K] of type a_type, B [N, K] E4M3, scales of both
// UE8M0 or FP32, B's per 1 << b_shift rows (0 or 7). With glu, B is the
// stacked [W_gate; W_up] and N = I, the activation's columns.
struct Fp8GemmArgs {
  const uint8_t* A;
  const void* As;
  const uint8_t* B;
  const void* Bs;
  int M, N, K;
  int kblocks;  // ceil(K / 128)
  int b_shift;
  void* C;        // the product [M, N]; with glu act, BF16 [M, I] (or null)
  uint16_t* gu;   // with glu: g and u, BF16 [M, 2 I], or null
};
enum Fp8Out { kFp8Bf16 = 0, kFp8F32 = 1, kFp8Glu = 2 };
// Whether either operand has fewer than four bytes of UE8M0 scales (the kernels
// read four at a time; launch_gemm_fp8_small takes these products too).
inline bool fp8_short_scales(int64_t M, int64_t N, int64_t kblocks, int b_shift) {
  return M * kblocks < 4 || ((N + (int64_t(1) << b_shift) - 1) >> b_shift) * kblocks < 4;
}
hipError_t launch_gemm_fp8_small(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type, bool scale_f32,
                                 hipStream_t stream);

// BF16 results and kFp8Glu (with its quantize) of UE8M0 operands, on 256 x 256
// tiles.
struct Fp8ActOut {
  uint8_t* codes;   // [M, I]
  uint8_t* scales;  // [M, I / 128]
};
hipError_t launch_gemm_fp8_tile(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type,
                                const Fp8ActOut& act, hipStream_t stream);

hipError_t launch_gemm_fp8(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type, bool scale_f32,
                           hipStream_t stream);

// Whether the gate+up product of these sizes runs on the kernel for few rows,
// which leaves act in BF16 (workspace: 2 M I bytes, where a.C is null) for a
// quantize of its own.
bool gemm_fp8_swiglu_small(int64_t M, int64_t I, int64_t K);
hipError_t launch_gemm_fp8_swiglu(const Fp8GemmArgs& a, uint8_t* codes, uint8_t* scales,
                                  void* workspace, hipStream_t stream);

// dact [M, I], gu [M, 2 I] BF16; codes [M, 2 I], scales [M, 2 I / 128], codes_t
// [2 I, Mp], scales_t [2 I, ceil(M / 128)], Mp = M rounded up to 16.
struct SwigluBackwardArgs {
  const uint16_t* dact;
  const uint16_t* gu;
  int M, I;
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* codes_t;
  uint8_t* scales_t;
};
hipError_t launch_swiglu_fp8_backward(const SwigluBackwardArgs& a, Fp8Type type,
                                      hipStream_t stream);

}  // namespace mxfp4
