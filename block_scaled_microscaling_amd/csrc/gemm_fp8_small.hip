// FP8 GEMM for few rows of A, and for few tiles: C[m, n] = sum over blocks
// kb of 128 of sa[m, kb] sb[n, kb] sum_k a[m, k] b[n, k], or the gate+up
// product of a gated MLP with act = silu(g) u. Decode-shaped: what bounds it
// is streaming B from HBM once, and with more rows reading A and B from L2.
//
// Work split. A workgroup of 8 waves owns 16 kMT rows of A and 16 kNT rows of
// B (kGlu: of gate and of up each); the blocks of K are dealt to its waves in
// turn, up to four neighbours at a time, so that even one row of A gives N / 16
// workgroups of eight waves, and the partial sums are added in LDS in the order
// of the waves.
//
// Data movement. An instruction loads 8 rows of 128 bytes, whole lines, into
// registers; a wave turns them into fragments through LDS of its own, where a
// row's eight 16-byte chunks are XOR-swizzled by the row. (Loading fragments, 16
// rows of 64 bytes an instruction, took 40 us instead of 29 for 128 x 8192 x
// 8192: the other half of each line is fetched again.) Loads are buffer loads
// whose resource ends behind the tile's last row: rows past M or N, blocks past
// K and the part of the last block past K give zeros and fetch nothing, so the
// next block's loads go out without a branch. One block ahead and two workgroups
// a CU did better than four blocks and fewer registers' worth of waves (1 x 8192
// x 8192 12.6 against 14.9 us). Four neighbouring blocks have their
// UE8M0 scales in one word: a load of one byte a row costs as much as one of
// the codes.
//
// Arithmetic. The codes go to BF16, exact, and through v_mfma_f32_16x16x32
// (fp8.h): memory bounds products of few rows, so the accuracy costs nothing.
// On 64 x 64 tiles, where it no longer does, BF16 results take the FP8
// v_mfma_scale_f32_16x16x128 (kBf16 false). UE8M0 scales are applied in the
// conversion or the instruction; FP32 scales multiply each block's sums: acc += (sa sb) * sums,
// B's scale the same for all of the tile's rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTileBytes = 16 * kFp8Block;  // 16 rows of one block
constexpr uint32_t kPast = 0x80000000u;  // an offset past every resource

// 16 rows of one block: lane l has chunk l % 8 of rows l / 8 and 8 + l / 8.
struct Lines {
  u32x4_t half[2];
};
__device__ __forceinline__ Lines load_lines(__amdgpu_buffer_rsrc_t rsrc, uint32_t at,
                                            uint32_t eight_rows, bool stream) {
  // (kPast plus any rows of a tile is past the resource as well.)
  Lines v;
  if (stream) {
    v.half[0] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)at, 0, kBufferNt);
    v.half[1] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)(at + eight_rows), 0, kBufferNt);
  } else {
    v.half[0] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)at, 0, 0);
    v.half[1] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)(at + eight_rows), 0, 0);
  }
  return v;
}

// Orders the LDS accesses of one wave's lanes among each other.
__device__ __forceinline__ void lds_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// v_mfma_f32_16x16x32_bf16: lane l holds 8 elements of K of row l % 16;
// accumulator register v of lane l holds (row of x) 4 (l / 16) + v, (row of y)
// l % 16.
__device__ __forceinline__ v4f_t mfma_bf16_16(bf16x8_t x, bf16x8_t y, v4f_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}

template <Fp8Type kA>
__device__ __forceinline__ v4f_t mfma_fp8_16(const v8i_t& x, const v8i_t& y, v4f_t c, uint32_t sx,
                                             uint32_t sy) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, kE4M3, kA, 0, (int)sx, 0,
                                                          (int)sy);
}

// One block of K of every tile of the workgroup, with its FP32 scales.
template <int kMT, int kNB>
struct Stage {
  Lines a[kMT], b[kNB];
  float sa[kMT], sb[kNB];
};
template <int kMT, int kNB>
struct Fragments {
  v8i_t a[kMT], b[kNB];
};

// Waves a SIMD that the registers must allow: two workgroups a CU where LDS has
// room.
template <int kMT, int kNB>
constexpr int kWavesOf = kMT + kNB <= 4 ? 4 : 2;

// kShort: a scale array of fewer than four bytes, which are loaded one by one.
template <int kMT, int kNT, Fp8Out kOut, Fp8Type kA, bool kF32Scale, bool kBf16, bool kStream,
          bool kShort>
__global__ __launch_bounds__(kThreads, (kWavesOf<kMT, (kOut == kFp8Glu ? 2 * kNT : kNT)>))
void gemm_fp8_small_kernel(Fp8GemmArgs p, int tiles_m, int tiles_n, int run) {
  constexpr bool kGlu = kOut == kFp8Glu;
  constexpr int kNB = kGlu ? 2 * kNT : kNT;
  // A wave's rows on their way into fragments; its sums at the end.
  constexpr int kPark = (kMT + kNB) * kTileBytes, kSums = kMT * kNB * 1024;
  __shared__ __align__(16) uint8_t lds[kWaves][kPark > kSums ? kPark : kSums];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  // The tiles of A that read the same rows of B run on one XCD (every 8th
  // workgroup), one behind the other.
  const int id = workgroup_id(tiles_m * tiles_n);
  if (id < 0) return;
  const int span = 8 * tiles_m;
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
  const uint32_t chunk = 16u * (lane & 7), row_at = (uint32_t)(lane >> 3) * K + chunk;

  // Rows of scales; rows past the end read the last one's. FP32: B's tiles lie
  // in one block of rows each, so its scale is the workgroup's.
  int64_t sa_at[kMT], sb_at[kNB];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
    sa_at[i] = (int64_t)min(m0 + 16 * i + r, p.M - 1) * p.kblocks;
#pragma unroll
  for (int j = 0; j < kNB; ++j) {
    const int n = min(n0 + 16 * (j % kNT) + (kF32Scale ? 0 : r), p.N - 1);
    // N is a multiple of 128 with kGlu: up's blocks begin behind gate's.
    sb_at[j] = (((j < kNT ? n : n + (int64_t)p.N)) >> p.b_shift) * p.kblocks;
  }
  const int64_t sa_total = (int64_t)p.M * p.kblocks;
  const int64_t b_rows = kGlu ? 2 * (int64_t)p.N : p.N;
  const int64_t sb_total = ((b_rows + (1 << p.b_shift) - 1) >> p.b_shift) * p.kblocks;

  // Block i of this wave's group g: `run` neighbours a wave, wave by wave.
  const auto block = [&](int g, int i) {
    return i < run ? (g * kWaves + wave) * run + i : p.kblocks;
  };
  const auto load = [&](Stage<kMT, kNB>& s, int kb) {
    const uint32_t k = (uint32_t)kb * kFp8Block;
    const uint32_t at = k + chunk < K ? row_at + k : kPast;
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      s.b[j] = load_lines(j < kNT ? rb : ru, at + (uint32_t)(16 * (j % kNT)) * K, 8 * K, kStream);
#pragma unroll
    for (int i = 0; i < kMT; ++i)
      s.a[i] = load_lines(ra, at + (uint32_t)(16 * i) * K, 8 * K, false);
    if constexpr (kF32Scale) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
        s.sa[i] = static_cast<const float*>(p.As)[sa_at[i] + min(kb, p.kblocks - 1)];
#pragma unroll
      for (int j = 0; j < kNB; ++j)
        s.sb[j] = static_cast<const float*>(p.Bs)[sb_at[j] + min(kb, p.kblocks - 1)];
    }
  };
  const auto word = [](const uint8_t* scales, int64_t at, int64_t total) {
    return kShort ? short_scale_word(scales, at, total) : scale_word(scales, at, total);
  };
  uint32_t wa[kMT], wb[kNB], na[kMT], nb[kNB];  // scale words of this group and the next
  const auto load_words = [&](int kb, uint32_t (&a)[kMT], uint32_t (&b)[kNB]) {
    if constexpr (!kF32Scale) {
      const int kc = min(kb, p.kblocks - 1);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
        a[i] = word(static_cast<const uint8_t*>(p.As), sa_at[i] + kc, sa_total);
#pragma unroll
      for (int j = 0; j < kNB; ++j)
        b[j] = word(static_cast<const uint8_t*>(p.Bs), sb_at[j] + kc, sb_total);
    }
  };

  // Through LDS: chunk c of row R lies at c ^ swizzle(R); lane l's fragment is
  // chunks l / 16 and 4 + l / 16 of row l % 16.
  uint8_t* mine = lds[wave];
  uint8_t* park_at[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = 8 * e + (lane >> 3);
    park_at[e] = mine + row * kFp8Block + 16 * ((lane & 7) ^ chunk_swizzle(row));
  }
  const uint8_t* frag_at[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    frag_at[e] = mine + r * kFp8Block + 16 * ((4 * e + q) ^ chunk_swizzle(r));
  const auto turn = [&](const Stage<kMT, kNB>& s) {
    Fragments<kMT, kNB> f;
#pragma unroll
    for (int t = 0; t < kMT + kNB; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<u32x4_t*>(park_at[e] + t * kTileBytes) =
            t < kNB ? s.b[t < kNB ? t : 0].half[e] : s.a[t < kNB ? 0 : t - kNB].half[e];
    lds_in_order();
#pragma unroll
    for (int t = 0; t < kMT + kNB; ++t) {
      const u32x4_t x = *reinterpret_cast<const u32x4_t*>(frag_at[0] + t * kTileBytes);
      const u32x4_t y = *reinterpret_cast<const u32x4_t*>(frag_at[1] + t * kTileBytes);
      (t < kNB ? f.b[t < kNB ? t : 0] : f.a[t < kNB ? 0 : t - kNB]) =
          (v8i_t){(int)x[0], (int)x[1], (int)x[2], (int)x[3],
                  (int)y[0], (int)y[1], (int)y[2], (int)y[3]};
    }
    lds_in_order();
    return f;
  };

  v4f_t acc[kMT][kNB];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = v4f_t{};

  const auto multiply = [&](const Fragments<kMT, kNB>& f, const float (&fa)[kMT],
                            const float (&fb)[kNB], int byte) {
    if constexpr (kBf16) {
      v4f_t sums[kMT][kNB];
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j) sums[i][j] = kF32Scale ? v4f_t{} : acc[i][j];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bf16x8_t a16[kMT], b16[kNB];
#pragma unroll
        for (int i = 0; i < kMT; ++i)
          a16[i] = fp8x8_to_bf16<kA>(
              (uint32_t)f.a[i][2 * k], (uint32_t)f.a[i][2 * k + 1],
              kF32Scale ? 1.0f : fp8_scale_value(wa[i] >> (8 * byte) & 255));
#pragma unroll
        for (int j = 0; j < kNB; ++j)
          b16[j] = fp8x8_to_bf16<kE4M3>(
              (uint32_t)f.b[j][2 * k], (uint32_t)f.b[j][2 * k + 1],
              kF32Scale ? 1.0f : fp8_scale_value(wb[j] >> (8 * byte) & 255));
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
          for (int j = 0; j < kNB; ++j) sums[i][j] = mfma_bf16_16(b16[j], a16[i], sums[i][j]);
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j) {
          if constexpr (kF32Scale) {
            const float scale = fa[i] * fb[j];
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(scale, sums[i][j][v], acc[i][j][v]);
          } else {
            acc[i][j] = sums[i][j];
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j) {
          if constexpr (kF32Scale) {
            const v4f_t d = mfma_fp8_16<kA>(f.b[j], f.a[i], v4f_t{}, 127, 127);
            const float scale = fa[i] * fb[j];
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(scale, d[v], acc[i][j][v]);
          } else {
            acc[i][j] = mfma_fp8_16<kA>(f.b[j], f.a[i], acc[i][j], wb[j] >> (8 * byte),
                                        wa[i] >> (8 * byte));
          }
        }
    }
  };

  Stage<kMT, kNB> s;
  load_words(block(0, 0), wa, wb);
  load(s, block(0, 0));
  for (int g = 0; block(g, 0) < p.kblocks; ++g) {
    load_words(block(g + 1, 0), na, nb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Fragments<kMT, kNB> f = turn(s);
      float fa[kMT], fb[kNB];
#pragma unroll
      for (int t = 0; t < kMT; ++t) fa[t] = s.sa[t];
#pragma unroll
      for (int t = 0; t < kNB; ++t) fb[t] = s.sb[t];
      load(s, i < 3 ? block(g, i + 1) : block(g + 1, 0));
      // (A block past the last is zeros, but its scales may be another row's.)
      if (block(g, i) < p.kblocks) multiply(f, fa, fb, i);
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i) wa[i] = na[i];
#pragma unroll
    for (int j = 0; j < kNB; ++j) wb[j] = nb[j];
  }

  // Lane l of tile (i, j) holds C[m0 + 16 i + l % 16][n0 + 16 j + 4 (l / 16) + v].
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      *reinterpret_cast<v4f_t*>(mine + (i * kNB + j) * 1024 + 16 * lane) = acc[i][j];
  __syncthreads();
  const auto sum = [&](int t) {
    v4f_t s = *reinterpret_cast<const v4f_t*>(lds[0] + t * 1024 + 16 * lane);
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
      s += *reinterpret_cast<const v4f_t*>(lds[w] + t * 1024 + 16 * lane);
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

template <int kMT, int kNT, Fp8Out kOut, Fp8Type kA, bool kF32Scale, bool kBf16 = true,
          bool kShort = false>
hipError_t launch(const Fp8GemmArgs& a, hipStream_t stream) {
  const int64_t tiles_m = ((int64_t)a.M + 16 * kMT - 1) / (16 * kMT);
  const int64_t tiles_n = ((int64_t)a.N + 16 * kNT - 1) / (16 * kNT);
  const dim3 grid = grid_of(tiles_m * tiles_n, kThreads);
  // Neighbouring blocks of a wave: four where K has that many for every wave.
  const int run = a.kblocks >= 4 * kWaves ? 4 : a.kblocks >= 2 * kWaves ? 2 : 1;
  // B's lines are read once where one tile of A covers all its rows.
  if (tiles_m == 1)
    hipLaunchKernelGGL(
        (gemm_fp8_small_kernel<kMT, kNT, kOut, kA, kF32Scale, kBf16, true, kShort>), grid,
        dim3(kThreads), 0, stream, a, (int)tiles_m, (int)tiles_n, run);
  else
    hipLaunchKernelGGL(
        (gemm_fp8_small_kernel<kMT, kNT, kOut, kA, kF32Scale, kBf16, false, kShort>), grid,
        dim3(kThreads), 0, stream, a, (int)tiles_m, (int)tiles_n, run);
  return hipGetLastError();
}

template <Fp8Out kOut, Fp8Type kA, bool kF32Scale>
hipError_t launch_sized(const Fp8GemmArgs& a, hipStream_t stream) {
  constexpr int kPair = kOut == kFp8Glu ? 2 : 1;  // gate and up tiles come in pairs
  constexpr int kTwo = 2 / kPair;
  if constexpr (!kF32Scale) {
    if (fp8_short_scales(a.M, kOut == kFp8Glu ? 2 * (int64_t)a.N : a.N, a.kblocks, a.b_shift))
      return launch<1, 1, kOut, kA, kF32Scale, true, true>(a, stream);
  }
  // One tile of rows where it holds all of A. More rows: the tile that reads A and
  // B least among those that leave no CU without a workgroup: 32 x 16 up to two
  // workgroups a CU (64 x 2048 x 4096 5.8 us against 11.4 with 64 x 32; 64 x 8192 x
  // 2048, past that, 12.3 against 9.7), 64 x 32 up to one (256 x 2048 x 4096 10.3
  // against 12.5 with 64 x 64; 256 x 4096 x 4096, past that, 18.9 against 13.0), or
  // two where 64 x 64 would be on BF16 instructions too (96 x 8192 x 8192 FP32 33.4
  // against 37.9). A tile of gate+up has twice the rows of B, so half as many do (64 x
  // 4096 x 2048 12.7 against 15.3; 64 x 4096 x 4096, past that, 22.8 against 16.7).
  const auto tiles = [&](int64_t m, int64_t n) { return (a.M + m - 1) / m * ((a.N + n - 1) / n); };
  if (a.M <= 16) return launch<1, 1, kOut, kA, kF32Scale>(a, stream);
  if (a.M <= 32 || tiles(32, 16) <= 512 / kPair)
    return launch<2, 1, kOut, kA, kF32Scale>(a, stream);
  if (a.M <= 64 || tiles(64, 16 * kTwo) <= (kOut == kFp8F32 ? 512 : 256 / kPair))
    return launch<4, kTwo, kOut, kA, kF32Scale>(a, stream);
  return launch<4, 2 * kTwo, kOut, kA, kF32Scale, kOut == kFp8F32>(a, stream);
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
