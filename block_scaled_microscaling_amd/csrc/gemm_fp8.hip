// FP8 GEMM on 128 x 128 tiles: C[m, n] = sum over blocks kb of 128 of
// sa[m, kb] sb[n, kb] sum_k a[m, k] b[n, k], in BF16 or FP32, or the gate+up
// product of a gated MLP with act = silu(g) u in BF16; and the choice of the
// kernel for every FP8 product.
//
// Tiling. A workgroup of 4 waves owns a 128 x 128 tile of C, wave (wy, wx) a 64
// x 64 part: 2 x 2 tiles of the 32 x 32 matrix instructions, B's fragment the
// first operand, so that a lane ends with four consecutive columns of one row.
// Two workgroups share a CU (64 KiB of LDS each), one computing while the
// other waits.
//
// Data movement. A K step is one block: 128 bytes a row, a whole line. Tiles go
// global -> LDS by DMA, 8 rows an instruction, one step ahead, in rows of eight
// 16-byte chunks XOR-swizzled by the row, so that a fragment's reads fall on
// all banks. Rows past M or N re-read the last one; chunks past K in a last
// step that is short come from a line of zeros (kTail).
//
// Arithmetic (fp8.h says why there are two):
//   FP8 codes straight into v_mfma_scale_f32_32x32x64_f8f6f4, or converted to
//   BF16 and through v_mfma_f32_32x32x16_bf16. UE8M0 scales go into the first
//   and into the conversion of the second; FP32 scales multiply each block's
//   sums (a lane holds one row of A, and B's scale is the wave's own), which
//   costs one FMA an element and block.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;                    // rows of A and of B per workgroup
constexpr int kRowBytes = kFp8Block;          // of one row in a K step
constexpr int kSlotBytes = kTile * kRowBytes;  // 16 KiB an operand
constexpr int kGroupM = 8;

typedef float v16_t __attribute__((ext_vector_type(16)));

// One block of K: codes of a 32-row tile, chunks h, 2 + h, 4 + h, 6 + h of the
// lane's row.
struct Frag {
  u32x4_t c[4];
};

template <Fp8Type kA, int kScaleOp>
__device__ __forceinline__ v16_t mfma_fp8_32(const Frag& x, const Frag& y, int s, v16_t c,
                                             uint32_t sx, uint32_t sy) {
  const u32x4_t x0 = x.c[2 * s], x1 = x.c[2 * s + 1], y0 = y.c[2 * s], y1 = y.c[2 * s + 1];
  const v8i_t xv = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3],
                    (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  const v8i_t yv = {(int)y0[0], (int)y0[1], (int)y0[2], (int)y0[3],
                    (int)y1[0], (int)y1[1], (int)y1[2], (int)y1[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xv, yv, c, kE4M3, kA, kScaleOp, (int)sx,
                                                         kScaleOp, (int)sy);
}

template <bool kBf16, bool kF32Scale, Fp8Out kOut, Fp8Type kA, bool kTail>
__global__ __launch_bounds__(kThreads, 2) void gemm_fp8_kernel(Fp8GemmArgs p, int tiles_m,
                                                               int tiles_n) {
  constexpr bool kGlu = kOut == kFp8Glu;
  __shared__ __align__(16) uint8_t lds[4 * kSlotBytes];  // slots 0, 1 of A, then of B

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wy = wave >> 1, wx = wave & 1;
  const int r = lane & 31, h = lane >> 5;
  const int id = workgroup_id(tiles_m * tiles_n);
  if (id < 0) return;
  int tm, tn;
  xcd_tile(id, tiles_m, tiles_n, kGroupM, tm, tn);
  const int row0 = tm * kTile;
  const int col0 = tn * (kGlu ? kTile / 2 : kTile);

  // B's row of tile row t. kGlu: a tile is 64 columns of act, wave column wx has
  // 32 of them, its first tile their gate rows, its second their up rows.
  const auto b_row = [&](int t) -> int64_t {
    if constexpr (kGlu)
      return (int64_t)min(col0 + 32 * (t >> 6) + (t & 31), p.N - 1) + ((t >> 5) & 1) * (int64_t)p.N;
    else
      return min(col0 + t, p.N - 1);
  };

  // This wave's DMAs: tile rows 32 w + 8 q + lane / 8 of each operand; lane l
  // lands at chunk l % 8 of its row and so fetches chunk (l % 8) ^ swizzle.
  const uint8_t* from_a[4];
  const uint8_t* from_b[4];
  int chunk[2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int t = 32 * wave + 8 * q + (lane >> 3);
    const int c = (lane & 7) ^ chunk_swizzle(t);
    if (q < 2) chunk[q] = c;  // the swizzle repeats every 16 rows
    from_a[q] = p.A + (int64_t)min(row0 + t, p.M - 1) * p.K + 16 * c;
    from_b[q] = p.B + b_row(t) * p.K + 16 * c;
  }
  const uint32_t lds0 = lds_addr(lds);
  const int last_bytes = p.K - (p.kblocks - 1) * kFp8Block;
  const auto load_step = [&](int kb, int slot) {
    const uint32_t to_a = __builtin_amdgcn_readfirstlane(lds0 + slot * kSlotBytes + wave * 4096);
    const uint32_t to_b = to_a + 2 * kSlotBytes;
    const int64_t k = (int64_t)kb * kRowBytes;
    const bool tail = kTail && kb == p.kblocks - 1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint8_t* ga = from_a[q] + k;
      const uint8_t* gb = from_b[q] + k;
      if (tail && 16 * chunk[q & 1] >= last_bytes) ga = gb = kFp8Zeros;
      dma16(ga, to_a + 1024 * q);
      dma16(gb, to_b + 1024 * q);
    }
  };

  // Scales. UE8M0: words of four blocks per row of the lane's tiles; FP32: the
  // next block's own.
  const int m_wave = row0 + 64 * wy;
  int64_t sa_at[2], sb_at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sa_at[i] = (int64_t)min(m_wave + 32 * i + r, p.M - 1) * p.kblocks;
    sb_at[i] = (b_row(64 * wx + 32 * i + (kF32Scale ? 0 : r)) >> p.b_shift) * p.kblocks;
  }
  const int64_t sa_total = (int64_t)p.M * p.kblocks;
  const int64_t b_rows = kGlu ? 2 * (int64_t)p.N : p.N;
  const int64_t sb_total = ((b_rows + (1 << p.b_shift) - 1) >> p.b_shift) * p.kblocks;
  uint32_t sa[2], sb[2];
  const auto load_scales = [&](int kb, uint32_t (&a)[2], uint32_t (&b)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (kF32Scale) {
        a[i] = static_cast<const uint32_t*>(p.As)[sa_at[i] + kb];
        b[i] = static_cast<const uint32_t*>(p.Bs)[sb_at[i] + kb];
      } else {
        a[i] = scale_word(static_cast<const uint8_t*>(p.As), sa_at[i] + kb, sa_total);
        b[i] = scale_word(static_cast<const uint8_t*>(p.Bs), sb_at[i] + kb, sb_total);
      }
    }
  };

  v16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v16_t{};

  const uint32_t x = (uint32_t)(h ^ chunk_swizzle(r));
  const uint8_t* frag_a = lds + (64 * wy + r) * kRowBytes;
  const uint8_t* frag_b = lds + 2 * kSlotBytes + (64 * wx + r) * kRowBytes;
  const auto read = [&](const uint8_t* base, int slot, int tile, Frag& f) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      f.c[c] = *reinterpret_cast<const u32x4_t*>(base + slot * kSlotBytes + tile * 32 * kRowBytes +
                                                 16 * ((2 * c) ^ x));
  };

  uint32_t na[2], nb[2];
  load_scales(0, na, nb);
  load_step(0, 0);
  for (int kb = 0; kb < p.kblocks; ++kb) {
    const int slot = kb & 1;
    // Every load of this step has landed, in all waves, and the other slot has
    // been read.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kF32Scale || (kb & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        asm volatile("" : "+v"(na[i]), "+v"(nb[i]));
        sa[i] = na[i];
        sb[i] = nb[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sa[i] >>= 8;
        sb[i] >>= 8;
      }
    }
    if (kb + 1 < p.kblocks) {
      if (kF32Scale || (kb & 3) == 3) load_scales(kb + 1, na, nb);
      load_step(kb + 1, 1 - slot);
    }
    Frag a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      read(frag_b, slot, i, b[i]);
      read(frag_a, slot, i, a[i]);
    }
    if constexpr (kBf16) {
      v16_t sums[2][2];
      if constexpr (kF32Scale) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) sums[i][j] = v16_t{};
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          bf16x8_t a16[2], b16[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t alo = a[i].c[c][2 * e], ahi = a[i].c[c][2 * e + 1];
            const uint32_t blo = b[i].c[c][2 * e], bhi = b[i].c[c][2 * e + 1];
            a16[i] = fp8x8_to_bf16<kA>(alo, ahi, kF32Scale ? 1.0f : fp8_scale_value(sa[i] & 255));
            b16[i] =
                fp8x8_to_bf16<kE4M3>(blo, bhi, kF32Scale ? 1.0f : fp8_scale_value(sb[i] & 255));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              v16_t& to = kF32Scale ? sums[i][j] : acc[i][j];
              to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b16[j], a16[i], to, 0, 0, 0);
            }
        }
      }
      if constexpr (kF32Scale) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = __uint_as_float(sa[i]) * __uint_as_float(sb[j]);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(f, sums[i][j][v], acc[i][j][v]);
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (kF32Scale) {
            v16_t s = mfma_fp8_32<kA, 0>(b[j], a[i], 0, v16_t{}, 127, 127);
            s = mfma_fp8_32<kA, 0>(b[j], a[i], 1, s, 127, 127);
            const float f = __uint_as_float(sa[i]) * __uint_as_float(sb[j]);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(f, s[v], acc[i][j][v]);
          } else {
            acc[i][j] = mfma_fp8_32<kA, 0>(b[j], a[i], 0, acc[i][j], sb[j], sa[i]);
            acc[i][j] = mfma_fp8_32<kA, 0>(b[j], a[i], 1, acc[i][j], sb[j], sa[i]);
          }
        }
    }
  }
  __syncthreads();

  // Register 4 q + t of tile (i, j) holds row 32 i + r, column 32 j + 8 q + 4 h
  // + t of the wave's part. Each wave parks it in its own 16 KiB and stores
  // whole lines: FP32 rows of 64 columns as 256 bytes, 16-byte chunk c at c ^
  // (row % 16); BF16 rows of `width` columns as 128 bytes, chunk c at c ^ (row
  // % 8).
  uint8_t* park = lds + wave * kSlotBytes;
  const int rows_left = p.M - m_wave;
  const auto store_bf16 = [&](uint16_t* to, int64_t ld, int cols, int width) {
    // to: the wave's first element; cols: how many columns there are
    const int lanes = width / 8;  // of a row
    if (ld % 8 == 0) {
      for (int x0 = 0; x0 < 64; x0 += 64 / lanes) {
        const int row = x0 + lane / lanes, c = lane % lanes;
        const u32x4_t v =
            *reinterpret_cast<const u32x4_t*>(park + row * 128 + 16 * (c ^ (row & 7)));
        if (row < rows_left && 8 * c < cols)
          *reinterpret_cast<u32x4_t*>(to + row * ld + 8 * c) = v;
      }
    } else {
      for (int row = 0; row < min(64, rows_left); ++row) {
        const uint16_t v = *reinterpret_cast<const uint16_t*>(
            park + row * 128 + 16 * ((lane >> 3) ^ (row & 7)) + 2 * (lane & 7));
        if (lane < cols) to[row * ld + lane] = v;
      }
    }
  };
  const auto park_bf16 = [&](int row, int col, uint32_t lo, uint32_t hi) {
    *reinterpret_cast<uint2*>(park + row * 128 + 16 * ((col >> 3) ^ (row & 7)) +
                              2 * (col & 7)) = make_uint2(lo, hi);
  };
  if constexpr (kGlu) {
    const int ncol = col0 + 32 * wx;
    uint16_t* act = static_cast<uint16_t*>(p.C) + (int64_t)m_wave * p.N + ncol;
    for (int part = p.gu ? 0 : 2; part < 3; ++part) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float g = acc[i][0][4 * q + t], u = acc[i][1][4 * q + t];
            v[t] = part == 0 ? g : part == 1 ? u : silu_f32(g) * u;
          }
          park_bf16(32 * i + r, 8 * q + 4 * h, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
      if (part == 2)
        store_bf16(act, p.N, 32, 32);
      else
        store_bf16(p.gu + (int64_t)m_wave * 2 * p.N + part * (int64_t)p.N + ncol,
                   2 * (int64_t)p.N, 32, 32);
    }
  } else if constexpr (kOut == kFp8Bf16) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v16_t& v = acc[i][j];
          park_bf16(32 * i + r, 32 * j + 8 * q + 4 * h, pack_bf16x2(v[4 * q], v[4 * q + 1]),
                    pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
        }
    const int ncol = col0 + 64 * wx;
    store_bf16(static_cast<uint16_t*>(p.C) + (int64_t)m_wave * p.N + ncol, p.N, p.N - ncol, 64);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v16_t& v = acc[i][j];
          const int c = 8 * j + 2 * q + h, row = 32 * i + r;
          *reinterpret_cast<float4*>(park + row * 256 + 16 * (c ^ (row & 15))) =
              make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
    const int ncol = col0 + 64 * wx, cols = p.N - ncol;
    float* to = static_cast<float*>(p.C) + (int64_t)m_wave * p.N + ncol;
    if (p.N % 4 == 0) {
      for (int x0 = 0; x0 < 64; x0 += 4) {
        const int row = x0 + (lane >> 4), c = lane & 15;
        const float4 v = *reinterpret_cast<const float4*>(park + row * 256 + 16 * (c ^ (row & 15)));
        if (row < rows_left && 4 * c < cols)
          *reinterpret_cast<float4*>(to + (int64_t)row * p.N + 4 * c) = v;
      }
    } else {
      for (int row = 0; row < min(64, rows_left); ++row) {
        const float v = *reinterpret_cast<const float*>(
            park + row * 256 + 16 * ((lane >> 2) ^ (row & 15)) + 4 * (lane & 3));
        if (lane < cols) to[(int64_t)row * p.N + lane] = v;
      }
    }
  }
}

template <bool kBf16, bool kF32Scale, Fp8Out kOut, Fp8Type kA>
hipError_t launch(const Fp8GemmArgs& a, hipStream_t stream) {
  constexpr int kCols = kOut == kFp8Glu ? kTile / 2 : kTile;
  const int64_t tiles_m = ((int64_t)a.M + kTile - 1) / kTile;
  const int64_t tiles_n = ((int64_t)a.N + kCols - 1) / kCols;
  const dim3 grid = grid_of(tiles_m * tiles_n, kThreads);
  if (a.K % kFp8Block != 0)
    hipLaunchKernelGGL((gemm_fp8_kernel<kBf16, kF32Scale, kOut, kA, true>), grid, dim3(kThreads),
                       0, stream, a, (int)tiles_m, (int)tiles_n);
  else
    hipLaunchKernelGGL((gemm_fp8_kernel<kBf16, kF32Scale, kOut, kA, false>), grid, dim3(kThreads),
                       0, stream, a, (int)tiles_m, (int)tiles_n);
  return hipGetLastError();
}

template <Fp8Type kA>
hipError_t launch_typed(const Fp8GemmArgs& a, Fp8Out out, bool f32, hipStream_t stream) {
  if (out == kFp8F32)
    return f32 ? launch<true, true, kFp8F32, kA>(a, stream)
               : launch<true, false, kFp8F32, kA>(a, stream);
  return f32 ? launch<false, true, kFp8Bf16, kA>(a, stream)
             : launch<false, false, kFp8Bf16, kA>(a, stream);
}

constexpr int kSmallMaxM = 512;

// Whether a product runs on 256 x 256 tiles: where they fill the chip.
bool big_tiles(int64_t M, int64_t N) {
  return M > 256 && ((M + 255) / 256) * ((N + 255) / 256) > 128;
}

}  // namespace

hipError_t launch_gemm_fp8(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type, bool scale_f32,
                           hipStream_t stream) {
  if (a.M <= kSmallMaxM || (!scale_f32 && fp8_short_scales(a.M, a.N, a.kblocks, a.b_shift)))
    return launch_gemm_fp8_small(a, out, a_type, scale_f32, stream);
  if (out == kFp8Bf16 && !scale_f32 && big_tiles(a.M, a.N))
    return launch_gemm_fp8_tile(a, out, a_type, Fp8ActOut{}, stream);
  return a_type == kE4M3 ? launch_typed<kE4M3>(a, out, scale_f32, stream)
                         : launch_typed<kE5M2>(a, out, scale_f32, stream);
}

bool gemm_fp8_swiglu_small(int64_t M, int64_t I, int64_t K) {
  return !big_tiles(M, 2 * I) || fp8_short_scales(M, 2 * I, (K + kFp8Block - 1) / kFp8Block, 7);
}

hipError_t launch_gemm_fp8_swiglu(const Fp8GemmArgs& a, uint8_t* codes, uint8_t* scales,
                                  void* workspace, hipStream_t stream) {
  if (!gemm_fp8_swiglu_small(a.M, a.N, a.K))
    return launch_gemm_fp8_tile(a, kFp8Glu, kE4M3, Fp8ActOut{codes, scales}, stream);
  Fp8GemmArgs g = a;
  if (!g.C) g.C = workspace;
  const hipError_t e = a.M <= kSmallMaxM || fp8_short_scales(a.M, 2 * (int64_t)a.N, a.kblocks, 7)
                           ? launch_gemm_fp8_small(g, kFp8Glu, kE4M3, false, stream)
                           : launch<false, false, kFp8Glu, kE4M3>(g, stream);
  if (e != hipSuccess) return e;
  Fp8QuantArgs q{};
  q.x = static_cast<const uint16_t*>(g.C);
  q.ldx = g.N;
  q.M = g.M;
  q.K = g.N;
  q.codes = codes;
  q.scales = scales;
  return launch_quantize_fp8(q, 1, kE4M3, stream);
}

}  // namespace mxfp4
