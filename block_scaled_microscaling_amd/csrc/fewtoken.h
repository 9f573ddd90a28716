// Shared by the few-token kernels (gemv.hip, moe.hip): products of MXFP4
// weight rows with a few activation rows, and the launchers that
// api_fewtoken.hip calls.
//
// One activation row: 64 lanes stream whole lines of a weight row and
// multiply their blocks on the VALU. Several: few_stream, on
// v_mfma_f32_16x16x32_bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gfx950.h"

namespace mxfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));

constexpr int kFewTile = 16;     // weight rows and activation rows of one MFMA
constexpr int kMaxWaves = 8;     // of a workgroup whose waves are segments of K
constexpr int kMaxPairs = 1024;  // T top_k of moe: its kernels' list of pairs is in LDS

__device__ __forceinline__ float scale_of_byte(uint32_t byte) {
  return __uint_as_float(byte << 23);
}

// Eight E2M1 codes (element 2i in bits 3:0 of byte i) times 2^(byte - 127),
// in BF16, exact; scale carries the UE8M0 byte in its float exponent field.
__device__ __forceinline__ bf16x8_t decode8(uint32_t w, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return (bf16x8_t){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <bool kOutFp32>
__device__ __forceinline__ void store_y(void* y, int64_t at, float v) {
  if constexpr (kOutFp32)
    static_cast<float*>(y)[at] = v;
  else
    static_cast<uint16_t*>(y)[at] = (uint16_t)pack_bf16x2(v, v);
}

// Orders the LDS accesses of one wave's lanes among each other.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------ one activation row
// Sums of two values over pairs of 16 lanes: a's in the even ones, b's in the
// odd ones.
__device__ __forceinline__ float merge16(float a, float b) {
  const auto s =
      __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// The sum over each 16 lanes, in all of them.
__device__ __forceinline__ float sum16(float sum) {
  const auto rotated = [](float f, auto ctrl) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(f), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  sum += rotated(sum, std::integral_constant<int, 0x128>{});
  sum += rotated(sum, std::integral_constant<int, 0x124>{});
  sum += rotated(sum, std::integral_constant<int, 0x122>{});
  sum += rotated(sum, std::integral_constant<int, 0x121>{});
  return sum;
}

// Lane sums of four rows -> the row r's total in lanes 16 r .. 16 r + 15.
__device__ __forceinline__ float sum_four_rows(const float (&v)[4]) {
  const auto merge32 = [](float a, float b) {  // low half: a's, high half: b's
    const auto s =
        __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
  };
  return sum16(merge16(merge32(v[0], v[2]), merge32(v[1], v[3])));
}

// Short rows, of up to kLanes (16, 32 or 64) blocks: a wave takes 64 / kLanes
// rows at a time, so that its lanes have work, and a workgroup is four waves
// that need nothing of each other.
constexpr int kShortWaves = 4;

// acc + the product of a block's 32 codes with 32 BF16 activations.
__device__ __forceinline__ float dot_block(u32x4_t w, float scale, const u32x4_t (&x)[4],
                                           float acc) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t ww = w[q], x0 = x[q][0], x1 = x[q][1], x2 = x[q][2], x3 = x[q][3];
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww, scale, 0),
                                          as_bf16x2(x0), acc, false);
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww, scale, 1),
                                          as_bf16x2(x1), acc, false);
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww, scale, 2),
                                          as_bf16x2(x2), acc, false);
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww, scale, 3),
                                          as_bf16x2(x3), acc, false);
  }
  return acc;
}

// The product of a block's 32 codes with 32 FP32 activations.
__device__ __forceinline__ float dot_block_f32(u32x4_t w, float scale, const u32x4_t (&a)[8]) {
  float dot = 0.0f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t ww = w[q];
    const v4f_t a0 = __builtin_bit_cast(v4f_t, a[2 * q]);
    const v4f_t a1 = __builtin_bit_cast(v4f_t, a[2 * q + 1]);
    const f32x2_t d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ww, scale, 0);
    const f32x2_t d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ww, scale, 1);
    const f32x2_t d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ww, scale, 2);
    const f32x2_t d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ww, scale, 3);
    dot = fmaf(d0[0], a0[0], dot);
    dot = fmaf(d0[1], a0[1], dot);
    dot = fmaf(d1[0], a0[2], dot);
    dot = fmaf(d1[1], a0[3], dot);
    dot = fmaf(d2[0], a1[0], dot);
    dot = fmaf(d2[1], a1[1], dot);
    dot = fmaf(d3[0], a1[2], dot);
    dot = fmaf(d3[1], a1[3], dot);
  }
  return dot;
}

// A wave's LDS for the activations of 64 blocks of kWords 16-byte words each:
// filled as whole lines (lane l has words l, l + 64, ...), read back a block a
// lane. The stride is odd in words, so that no reads meet on a bank.
template <int kWords>
struct LaneBlocks {
  static constexpr int kStride = (kWords | 1) * 16;
  static constexpr int kBytes = 64 * kStride;
  static __device__ __forceinline__ void fill(uint8_t* lds, const u32x4_t (&r)[kWords]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int at = i * 64 + lane;
      *reinterpret_cast<u32x4_t*>(lds + at / kWords * kStride + at % kWords * 16) = r[i];
    }
    wave_sync();
  }
  static __device__ __forceinline__ u32x4_t get(const uint8_t* lds, int i) {
    return *reinterpret_cast<const u32x4_t*>(lds + (threadIdx.x & 63) * kStride + i * 16);
  }
};

// --------------------------------------------------- several activation rows
// Work of a wave: units of 256 k (8 blocks) of T tiles of 16 weight rows and
// of up to 16 activation columns. Everything is fetched as whole lines (8
// weight rows x 128 B an instruction, X's activations alike), parked in the
// wave's own LDS and read back as the MFMA's fragments: lane l has row l %
// 16's dword l / 16 of a block (8 codes) and the same 8 k of activation
// column l % 16, so accumulator register v of lane l is output (weight row
// 4 (l / 16) + v, column l % 16).
// Loading fragments straight from the rows touches 16 to 32 lines an
// instruction: 8 x 4096 x 14336 12.0 us against 8.6 us, 16 x 8192 x 8192 12.6
// against 10.9 us. With kAhead a unit is loaded while the last one is used;
// without, its registers make room for more waves. Two to four units ahead
// were no faster at any shape, nor were tiles sharing the activations'
// fragments in registers (16 x 28672 x 4096 17.0 us, 16 x 8192 x 8192 12.1).
constexpr int kUnitBlocks = 8;
constexpr int kXStride = 256 + 16;  // LDS row strides: padded, so that the
constexpr int kWStride = 128 + 16;  // fragment reads meet no bank conflicts

// Activations for few_stream: 4 XL BF16 rows, one a column, whose blocks start
// kBlockBytes apart. Lane l loads rows 4 i + l / 16, 16 bytes each.
template <int XL, int kBlockBytes = 64>
struct BfRows {
  static constexpr int kColumns = 4 * XL;
  struct Half {
    u32x4_t r[XL];
  };
  const uint8_t* p[XL];  // the lane's rows, with its place (l % 4) in a block

  // Half h (128 k) of unit u; blocks past the row are read as its last.
  __device__ __forceinline__ void load(Half& a, int u, int h, int KB) const {
    const int b = min(u * kUnitBlocks + h * 4 + (int)((threadIdx.x & 15) >> 2), KB - 1);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      a.r[i] = *reinterpret_cast<const u32x4_t*>(p[i] + (int64_t)b * kBlockBytes);
  }
  // Zeros in place of the blocks from nb of the unit.
  __device__ __forceinline__ void cut(Half& a, int h, int nb) const {
    if (h * 4 + (int)((threadIdx.x & 15) >> 2) >= nb) {
#pragma unroll
      for (int i = 0; i < XL; ++i) a.r[i] = u32x4_t{0u, 0u, 0u, 0u};
    }
  }
  __device__ __forceinline__ void park(const Half& a, uint8_t* lds) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < XL; ++i)
      *reinterpret_cast<u32x4_t*>(lds + (4 * i + (lane >> 4)) * kXStride + (lane & 15) * 16) =
          a.r[i];
  }
};

template <int T, class X>
constexpr int few_lds_bytes() {  // per wave
  return X::kColumns * kXStride + T * kFewTile * kWStride;
}

// Adds to acc the products over the units first, first + stride, ... of rows
// row(t, 0 .. 15), counted from codes[t] and scales[t] (KB blocks a row; both
// pointers the same in every lane, the rows' bytes within 2^32 of them).
template <int T, bool kAhead, class X, class Row>
__device__ __forceinline__ void few_stream(const uint8_t* const (&codes)[T],
                                           const uint8_t* const (&scales)[T], const Row& row,
                                           const X& x, int KB, int first, int stride, uint8_t* lds,
                                           v4f_t (&acc)[T]) {
  const int lane = threadIdx.x & 63;
  const int a = lane & 15, g = lane >> 4, blk = lane & 7;
  const int column = min(a, X::kColumns - 1);
  uint8_t* xl = lds;
  uint8_t* wl = lds + X::kColumns * kXStride;
  uint32_t cp[T][2], sp[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
#pragma unroll
    for (int d = 0; d < 2; ++d) cp[t][d] = (uint32_t)row(t, 8 * d + (lane >> 3)) * KB * 16;
    sp[t] = (uint32_t)row(t, a) * KB;
  }
  const int units = (KB + kUnitBlocks - 1) / kUnitBlocks;
  if (first >= units) return;
  u32x4_t w[T][2];
  uint64_t sc[T];
  typename X::Half xr[2];

  // Blocks past the row are read as its last and taken as zeros when used.
  // The eight scale bytes are those that end with the row's last.
  const auto load = [&](int u) {
    const uint32_t at = (uint32_t)min(u * kUnitBlocks + blk, KB - 1) * 16;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int d = 0; d < 2; ++d)
        w[t][d] = *reinterpret_cast<const u32x4_t*>(codes[t] + (cp[t][d] + at));
    if (KB >= kUnitBlocks) {
      const uint32_t from = (uint32_t)min(u * kUnitBlocks, KB - kUnitBlocks);
#pragma unroll
      for (int t = 0; t < T; ++t) __builtin_memcpy(&sc[t], scales[t] + (sp[t] + from), 8);
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        sc[t] = 0;
        for (int i = 0; i < KB; ++i)
          sc[t] |= (uint64_t)scales[t][sp[t] + i] << (8 * (kUnitBlocks - KB + i));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) x.load(xr[h], u, h, KB);
  };

  if (kAhead) load(first);
  for (int u = first; u < units; u += stride) {
    if (!kAhead) load(u);
    const int nb = KB - u * kUnitBlocks;
    uint64_t cs[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int d = 0; d < 2; ++d)
        *reinterpret_cast<u32x4_t*>(wl + (t * kFewTile + 8 * d + (lane >> 3)) * kWStride +
                                    blk * 16) = w[t][d];
      cs[t] = sc[t];
    }
    if (nb < kUnitBlocks) {
      // Scale 1 and activations of zero for what is past the row.
#pragma unroll
      for (int t = 0; t < T; ++t)
        cs[t] = (cs[t] >> (8 * (kUnitBlocks - nb))) | (0x7F7F7F7F7F7F7F7Full << (8 * nb));
#pragma unroll
      for (int h = 0; h < 2; ++h) x.cut(xr[h], h, nb);
    }
    x.park(xr[0], xl);
    const typename X::Half x1 = xr[1];
    if (kAhead && u + stride < units) load(u + stride);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1) {
        wave_sync();
        x.park(x1, xl);
      }
      wave_sync();
      bf16x8_t xf[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        xf[b] = *reinterpret_cast<const bf16x8_t*>(xl + column * kXStride + b * 64 + g * 16);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint32_t c4 = (uint32_t)(cs[t] >> (32 * h));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t ww = *reinterpret_cast<const uint32_t*>(
              wl + (t * kFewTile + a) * kWStride + (4 * h + b) * 16 + 4 * g);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              decode8(ww, scale_of_byte((c4 >> (8 * b)) & 0xFF)), xf[b], acc[t], 0, 0, 0);
        }
      }
    }
    wave_sync();
  }
}

// The next BF16 piece of v, which becomes its rest: the first 8 bits of the
// significand, the rest being exact, so three pieces are all 24. Cut and not
// rounded: FP32 values next to the largest would round to infinity. (Bits below
// BF16's least, 2^-133, are lost: of values under 2^-109.)
__device__ __forceinline__ uint16_t next_piece(float& v) {
  const uint32_t bits = __float_as_uint(v) & 0xFFFF0000u;
  // No rest where the piece is no finite number: inf - inf is NaN.
  v = (bits & 0x7F800000u) == 0x7F800000u ? 0.0f : v - __uint_as_float(bits);
  return (uint16_t)(bits >> 16);
}

// Products for workgroups whose waves share x: waves are kShareTiles tiles of
// 16 weight rows times `parts` parts of K. The four waves of a part load a
// quarter each of a unit of its 4 XL rows of x into LDS. Up to 16 rows are
// double-buffered, with one barrier a unit; for 32 that LDS would cost waves.
constexpr int kShareTiles = 4;
constexpr int kShareStride = 512 + 16;  // LDS row stride of a unit of x, padded

// An LDS barrier of the workgroup that leaves global loads in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int XL>
constexpr int share_x_bytes() {  // of one part of K
  return (XL > 4 ? 1 : 2) * 4 * XL * kShareStride;
}

template <int XL>
constexpr int share_lds_bytes(int parts) {
  return parts * (share_x_bytes<XL>() + kShareTiles * kFewTile * kWStride);
}

// Adds to acc the products of weight rows row(0 .. 15), counted from codes and
// scales (KB blocks a row, within 2^32 bytes), with the rows of x at xrow(0 ..
// 4 XL - 1), given with the lane's place (lane % 4) in a block and blocks that
// start kBlockBytes apart, over the units part, part + parts, ...; tile is the
// wave's in its part. Column c of x's rows is column c % 16 of acc[c / 16].
template <int XL, int kBlockBytes, class Row, class XRow>
__device__ __forceinline__ void share_stream(const uint8_t* codes, const uint8_t* scales,
                                             const Row& row, const XRow& xrow, int KB, int tile,
                                             int part, int parts, uint8_t* lds,
                                             v4f_t (&acc)[(XL + 3) / 4]) {
  // Pieces of a unit of x: 4 rows x 256 bytes, one load of a wave each.
  constexpr int kColumns = 4 * XL, kPieces = 2 * XL, kGroups = (XL + 3) / 4;
  constexpr int kMine = (kPieces + kShareTiles - 1) / kShareTiles;
  constexpr bool kTwoBuffers = XL <= 4;
  constexpr int kBuffer = kTwoBuffers ? kColumns * kShareStride : 0;
  const int lane = threadIdx.x & 63;
  const int a = lane & 15, g = lane >> 4, blk = lane & 7;
  uint8_t* xl = lds + part * share_x_bytes<XL>();
  uint8_t* wl =
      lds + parts * share_x_bytes<XL>() + (part * kShareTiles + tile) * kFewTile * kWStride;
  const int column = min(a, kColumns - 1);
  const int units = (KB + kUnitBlocks - 1) / kUnitBlocks;
  uint32_t cp[2];
#pragma unroll
  for (int d = 0; d < 2; ++d) cp[d] = (uint32_t)row(8 * d + (lane >> 3)) * KB * 16;
  const uint32_t sp = (uint32_t)row(a) * KB;
  const uint8_t* xp[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    xp[i] = xrow((4 * ((tile + i * kShareTiles) >> 1) + g) % kColumns);
  u32x4_t w[2], xr[kMine];
  uint64_t sc, cs = 0;
  const auto load = [&](int u) {
    const uint32_t at = (uint32_t)min(u * kUnitBlocks + blk, KB - 1) * 16;
#pragma unroll
    for (int d = 0; d < 2; ++d)
      w[d] = *reinterpret_cast<const u32x4_t*>(codes + (cp[d] + at));
    if (KB >= kUnitBlocks) {
      const uint32_t from = (uint32_t)min(u * kUnitBlocks, KB - kUnitBlocks);
      __builtin_memcpy(&sc, scales + (sp + from), 8);
    } else {
      sc = 0;
      for (int i = 0; i < KB; ++i)
        sc |= (uint64_t)scales[sp + i] << (8 * (kUnitBlocks - KB + i));
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int piece = tile + i * kShareTiles;
      if (piece >= kPieces) break;
      const int b = min(u * kUnitBlocks + (piece & 1) * 4 + (a >> 2), KB - 1);
      xr[i] = *reinterpret_cast<const u32x4_t*>(xp[i] + (int64_t)b * kBlockBytes);
    }
  };
  const auto park = [&](int u, int buffer) {
    // Blocks past the row: scale 1 and activations of zero.
    const int nb = KB - u * kUnitBlocks;
#pragma unroll
    for (int d = 0; d < 2; ++d)
      *reinterpret_cast<u32x4_t*>(wl + (8 * d + (lane >> 3)) * kWStride + blk * 16) = w[d];
    cs = sc;
    if (nb < kUnitBlocks)
      cs = (cs >> (8 * (kUnitBlocks - nb))) | (0x7F7F7F7F7F7F7F7Full << (8 * nb));
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int piece = tile + i * kShareTiles, half = piece & 1;
      if (piece >= kPieces) break;
      if (half * 4 + (a >> 2) >= nb) xr[i] = u32x4_t{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4_t*>(xl + buffer * kBuffer + (4 * (piece >> 1) + g) * kShareStride +
                                  half * 256 + a * 16) = xr[i];
    }
  };

  int u = part;
  if (u < units) {
    load(u);
    park(u, 0);
  }
  // Every wave meets every barrier, with or without a unit of its own. A
  // buffer is written again only after the barrier that follows its use.
  for (int i = 0; i * parts < units; ++i, u += parts) {
    if (u + parts < units) load(u + parts);
    lds_barrier();
    if (u < units) {
#pragma unroll
      for (int b = 0; b < kUnitBlocks; ++b) {
        const uint32_t ww = *reinterpret_cast<const uint32_t*>(wl + a * kWStride + b * 16 + 4 * g);
        const bf16x8_t wf = decode8(ww, scale_of_byte((uint32_t)(cs >> (8 * b)) & 0xFF));
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
          const bf16x8_t xf = *reinterpret_cast<const bf16x8_t*>(
              xl + (i & 1) * kBuffer + (16 * q + column) * kShareStride + b * 64 + g * 16);
          acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf, acc[q], 0, 0, 0);
        }
      }
      wave_sync();
    }
    if (!kTwoBuffers) lds_barrier();
    if (u + parts < units) park(u + parts, (i + 1) & 1);
  }
}

// Waves that share `items` evenly, of at most `most`.
inline int even_waves(int items, int most) {
  const int rounds = (items + most - 1) / most;
  return (items + rounds - 1) / rounds;
}

// Launchers: arguments are validated by the caller.
hipError_t launch_gemv(const void* x, int64_t ldx, const void* codes, const void* scales, int M,
                       int N, int K, bool out_fp32, void* y, hipStream_t stream);
int64_t moe_route_workspace_bytes(int64_t T, int64_t H, int64_t E);
hipError_t launch_moe_route(const void* x, int64_t ldx, const void* router, int T, int H, int E,
                            int top_k, bool renormalize, int32_t* ids, float* weights,
                            double* logits, hipStream_t stream);
hipError_t launch_moe(const void* x, int64_t ldx, const int32_t* ids, const float* weights,
                      const void* w13, const void* w13_s, const void* w2, const void* w2_s, int T,
                      int H, int I, int E, int top_k, bool out_fp32, void* y, void* workspace,
                      hipStream_t stream);

}  // namespace mxfp4
