// FP8 GEMM for few rows of A, and for few tiles: C[m, n] = sum over blocks
// kb of 128 of sa[m, kb] sb[n, kb] sum_k a[m, k] b[n, k], or the gate+up
// product of a gated MLP with act = silu(g) u. Decode-shaped: what bounds it
// is streaming B from HBM once.
//
// Work split. A workgroup of 8 waves owns 16 kMT rows of A and 16 kNT rows of
// B (kGlu: of gate and of up each); the blocks of K are dealt to its waves in
// turn, so that even one row of A gives N / 16 workgroups of eight waves, and
// the partial sums are added in LDS in the order of the waves.
//
// Data movement. Lane l loads 16-byte chunks l / 16 and 4 + l / 16 of its
// row's 128 bytes straight into registers: an instruction reads 16 rows of 64
// bytes. (A block has one scale, so which of its elements a lane holds does
// not matter as long as A and B agree.) Loads are buffer loads whose resource
// ends behind the tile's last row: rows past M or N, blocks past K and the
// part of the last block past K give zeros and fetch nothing, so loads run
// kDepth blocks ahead without a branch.
//
// Arithmetic. The codes go to BF16, exact, and through v_mfma_f32_16x16x32
// (fp8.h): memory bounds these products, so the accuracy costs nothing. UE8M0
// scales are applied in the conversion; FP32 scales multiply each block's
// sums: acc += (sa sb) * sums, B's scale the same for all of the tile's rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr uint32_t kPast = 0x80000000u;  // an offset past every resource

__device__ __forceinline__ v8i_t load_block(__amdgpu_buffer_rsrc_t rows, uint32_t row_at,
                                            uint32_t k, uint32_t K, bool stream) {
  const uint32_t o0 = k < K ? row_at + k : kPast;
  const uint32_t o1 = k + 64 < K ? row_at + k + 64 : kPast;
  u32x4_t a, b;
  if (stream) {
    a = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)o0, 0, kBufferNt);
    b = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)o1, 0, kBufferNt);
  } else {
    a = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)o0, 0, 0);
    b = __builtin_amdgcn_raw_buffer_load_b128(rows, (int)o1, 0, 0);
  }
  return (v8i_t){(int)a[0], (int)a[1], (int)a[2], (int)a[3],
                 (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

template <Fp8Type kType>
__device__ __forceinline__ void to_bf16(const v8i_t& v, float scale, bf16x8_t (&out)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    out[k] = fp8x8_to_bf16<kType>((uint32_t)v[2 * k], (uint32_t)v[2 * k + 1], scale);
}

// v_mfma_f32_16x16x32_bf16: lane l holds 8 elements of K of row l % 16;
// accumulator register v of lane l holds (row of x) 4 (l / 16) + v, (row of y)
// l % 16.
__device__ __forceinline__ v4f_t mfma_bf16_16(bf16x8_t x, bf16x8_t y, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}

// One block of K of every tile of the workgroup.
template <int kMT, int kNB>
struct Stage {
  v8i_t a[kMT], b[kNB];
  uint32_t sa[kMT], sb[kNB];  // UE8M0 bytes, or FP32 bits
};

template <int kMT, int kNT, Fp8Out kOut, Fp8Type kA, bool kF32Scale, bool kStream>
__global__ __launch_bounds__(kThreads) void gemm_fp8_small_kernel(Fp8GemmArgs p, int tiles_m,
                                                                  int tiles_n) {
  constexpr bool kGlu = kOut == kFp8Glu;
  constexpr int kNB = kGlu ? 2 * kNT : kNT;
  constexpr int kDepth = kMT + kNB <= 3 ? 4 : kMT + kNB <= 4 ? 3 : 2;
  __shared__ __align__(16) float red[kWaves][kMT * kNB][256];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  // The tiles of A that read the same rows of B run on one XCD (every 8th
  // workgroup), one behind the other.
  const int span = 8 * tiles_m;
  const int id = workgroup_id(tiles_m * tiles_n);
  if (id < 0) return;
  const int grp = id / span, in = id - grp * span;
  const int left = min(8, tiles_n - 8 * grp);
  const int tm = in / left, tn = 8 * grp + in - tm * left;
  const int m0 = 16 * kMT * tm, n0 = 16 * kNT * tn;

  const uint32_t K = (uint32_t)p.K;
  const int rows_a = min(16 * kMT, p.M - m0);
  const int rows_b = min(16 * kNT, p.N - n0);
  const auto resource = [](const uint8_t* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)bytes,
                                             kBufferWord3);
  };
  const auto ra = resource(p.A + (int64_t)m0 * K, (uint32_t)rows_a * K);
  const auto rb = resource(p.B + (int64_t)n0 * K, (uint32_t)rows_b * K);
  const auto ru = resource(p.B + ((int64_t)n0 + (kGlu ? p.N : 0)) * K, (uint32_t)rows_b * K);
  const uint32_t row_at = (uint32_t)r * K;

  // Rows of scales; rows past the end read the last one's.
  int64_t sa_at[kMT], sb_at[kNB];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
    sa_at[i] = (int64_t)min(m0 + 16 * i + r, p.M - 1) * p.kblocks;
#pragma unroll
  for (int j = 0; j < kNB; ++j) {
    const int n = min(n0 + 16 * (j % kNT) + r, p.N - 1);
    // N is a multiple of 128 with kGlu: up's blocks begin behind gate's.
    sb_at[j] = (int64_t)((j < kNT ? n : n + p.N) >> p.b_shift) * p.kblocks;
  }

  const auto load = [&](Stage<kMT, kNB>& s, int kb) {
    const uint32_t k = (uint32_t)kb * kFp8Block + 16u * q;
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      s.b[j] = load_block(j < kNT ? rb : ru, row_at + (uint32_t)(16 * (j % kNT)) * K, k, K,
                          kStream);
#pragma unroll
    for (int i = 0; i < kMT; ++i)
      s.a[i] = load_block(ra, row_at + (uint32_t)(16 * i) * K, k, K, false);
    const int kc = min(kb, p.kblocks - 1);
#pragma unroll
    for (int i = 0; i < kMT; ++i)
      s.sa[i] = kF32Scale ? static_cast<const uint32_t*>(p.As)[sa_at[i] + kc]
                          : static_cast<const uint8_t*>(p.As)[sa_at[i] + kc];
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      s.sb[j] = kF32Scale ? static_cast<const uint32_t*>(p.Bs)[sb_at[j] + kc]
                          : static_cast<const uint8_t*>(p.Bs)[sb_at[j] + kc];
  };

  v4f_t acc[kMT][kNB];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = v4f_t{};

  Stage<kMT, kNB> st[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load(st[d], wave + d * kWaves);
  for (int kb = wave; kb < p.kblocks; kb += kDepth * kWaves) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (kb + d * kWaves < p.kblocks) {
        bf16x8_t a16[kMT][4], b16[kNB][4];
#pragma unroll
        for (int i = 0; i < kMT; ++i)
          to_bf16<kA>(st[d].a[i], kF32Scale ? 1.0f : fp8_scale_value(st[d].sa[i]), a16[i]);
#pragma unroll
        for (int j = 0; j < kNB; ++j)
          to_bf16<kE4M3>(st[d].b[j], kF32Scale ? 1.0f : fp8_scale_value(st[d].sb[j]), b16[j]);
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
          for (int j = 0; j < kNB; ++j) {
            v4f_t s = kF32Scale ? v4f_t{} : acc[i][j];
#pragma unroll
            for (int k = 0; k < 4; ++k) s = mfma_bf16_16(b16[j][k], a16[i][k], s);
            if constexpr (kF32Scale) {
              const float f = __uint_as_float(st[d].sa[i]) * __uint_as_float(st[d].sb[j]);
#pragma unroll
              for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(f, s[v], acc[i][j][v]);
            } else {
              acc[i][j] = s;
            }
          }
      }
      load(st[d], kb + (d + kDepth) * kWaves);
    }
  }

  // Lane l of tile (i, j) holds C[m0 + 16 i + l % 16][n0 + 16 j + 4 (l / 16) + v].
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      *reinterpret_cast<v4f_t*>(&red[wave][i * kNB + j][4 * lane]) = acc[i][j];
  __syncthreads();
  const auto sum = [&](int t) {
    v4f_t s = *reinterpret_cast<const v4f_t*>(&red[0][t][4 * lane]);
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
      s += *reinterpret_cast<const v4f_t*>(&red[w][t][4 * lane]);
    return s;
  };
  for (int t = wave; t < kMT * kNT; t += kWaves) {
    const int i = t / kNT, j = t - i * kNT;
    const int m = m0 + 16 * i + r, n = n0 + 16 * j + 4 * q;
    v4f_t s = sum(i * kNB + j);
    if (m >= p.M || n >= p.N) continue;
    if constexpr (kGlu) {
      const v4f_t u = sum(i * kNB + kNT + j);
      if (p.gu) {
        uint16_t* g_at = p.gu + (int64_t)m * 2 * p.N + n;
        *reinterpret_cast<uint2*>(g_at) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
        *reinterpret_cast<uint2*>(g_at + p.N) =
            make_uint2(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) s[v] = silu_f32(s[v]) * u[v];
    }
    const int64_t at = (int64_t)m * p.N + n;
    if (p.N % 4 == 0) {
      if constexpr (kOut == kFp8F32)
        *reinterpret_cast<v4f_t*>(static_cast<float*>(p.C) + at) = s;
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + at) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (n + v >= p.N) break;
        if constexpr (kOut == kFp8F32)
          static_cast<float*>(p.C)[at + v] = s[v];
        else
          static_cast<uint16_t*>(p.C)[at + v] = (uint16_t)pack_bf16x2(s[v], s[v]);
      }
    }
  }
}

template <int kMT, int kNT, Fp8Out kOut, Fp8Type kA, bool kF32Scale>
hipError_t launch(const Fp8GemmArgs& a, hipStream_t stream) {
  const int64_t tiles_m = ((int64_t)a.M + 16 * kMT - 1) / (16 * kMT);
  const int64_t tiles_n = ((int64_t)a.N + 16 * kNT - 1) / (16 * kNT);
  const dim3 grid = grid_of(tiles_m * tiles_n, kThreads);
  // B's lines are read once where one tile of A covers all its rows.
  if (tiles_m == 1)
    hipLaunchKernelGGL((gemm_fp8_small_kernel<kMT, kNT, kOut, kA, kF32Scale, true>), grid,
                       dim3(kThreads), 0, stream, a, (int)tiles_m, (int)tiles_n);
  else
    hipLaunchKernelGGL((gemm_fp8_small_kernel<kMT, kNT, kOut, kA, kF32Scale, false>), grid,
                       dim3(kThreads), 0, stream, a, (int)tiles_m, (int)tiles_n);
  return hipGetLastError();
}

template <Fp8Out kOut, Fp8Type kA, bool kF32Scale>
hipError_t launch_sized(const Fp8GemmArgs& a, hipStream_t stream) {
  if (a.M <= 16) return launch<1, 1, kOut, kA, kF32Scale>(a, stream);
  if (a.M <= 32) return launch<2, 1, kOut, kA, kF32Scale>(a, stream);
  return launch<4, kOut == kFp8Glu ? 1 : 2, kOut, kA, kF32Scale>(a, stream);
}

template <Fp8Out kOut>
hipError_t launch_typed(const Fp8GemmArgs& a, Fp8Type a_type, bool f32, hipStream_t stream) {
  if (a_type == kE4M3)
    return f32 ? launch_sized<kOut, kE4M3, true>(a, stream)
               : launch_sized<kOut, kE4M3, false>(a, stream);
  return f32 ? launch_sized<kOut, kE5M2, true>(a, stream)
             : launch_sized<kOut, kE5M2, false>(a, stream);
}

}  // namespace

hipError_t launch_gemm_fp8_small(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type, bool scale_f32,
                                 hipStream_t stream) {
  if (out == kFp8Glu) return launch_sized<kFp8Glu, kE4M3, false>(a, stream);
  return out == kFp8F32 ? launch_typed<kFp8F32>(a, a_type, scale_f32, stream)
                        : launch_typed<kFp8Bf16>(a, a_type, scale_f32, stream);
}

}  // namespace mxfp4
