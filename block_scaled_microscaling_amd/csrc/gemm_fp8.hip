// FP8 GEMM on tiles of 128 x 128 or 128 x 256: C[m, n] = sum over blocks kb of
// 128 of sa[m, kb] sb[n, kb] sum_k a[m, k] b[n, k], in BF16 or FP32, or the
// gate+up product of a gated MLP with act = silu(g) u in BF16; and the choice of
// the kernel for every FP8 product.
//
// Tiling. One workgroup of 4 waves (one per SIMD) owns a tile of C, wave (wy, wx)
// 64 rows and 32 kNT columns of it: 2 x kNT tiles of the 32 x 32 matrix
// instructions, B's fragment the first operand, so that a lane ends with four
// consecutive columns of one row. With at most 128 accumulators a lane the
// vector registers hold them, which FP32 scales need: a block's sums times its
// scale are added on the VALU (on 256 x 256 tiles they would go to and from the
// accumulation registers, three instructions for one).
//
// Data movement. A K step is one block: 128 bytes a row, a whole line. Tiles and
// scales (one dword a row) go global -> LDS by DMA into a ring of kSlots slots,
// tiles in rows of eight 16-byte chunks XOR-swizzled by the row, so that a
// fragment's reads fall on all banks. The fragments of a step are read while the
// step before is multiplied, so a slot is free once its step begins, and loads
// run kSlots steps ahead. Every wave issues the same number of DMAs a step, and
// nothing else that counts with them; so a wait names how many may be under way.
// Rows past M or N re-read the last one; chunks past K in a last step that is
// short come from a line of zeros (kTail).
//
// Arithmetic (fp8.h says why there are two):
//   FP8 codes straight into v_mfma_scale_f32_32x32x64_f8f6f4, or converted to
//   BF16 and through v_mfma_f32_32x32x16_bf16. UE8M0 scales go into the first
//   and into the conversion of the second; FP32 scales multiply each block's
//   sums (a lane holds one row of A, and B's scale is the wave's own).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;            // of A per workgroup
constexpr int kRowBytes = kFp8Block;  // of one row in a K step
constexpr int kGroupM = 8;

// Columns of a tile, its LDS slot and ring, and the DMAs of a wave's step: 4 of
// A's rows, 2 kNT of B's, and 64 rows of scales (two of them with kNT = 4).
template <int kNT>
struct Geom {
  static constexpr int kCols = 64 * kNT;
  static constexpr int kTiles = (kRows + kCols) * kRowBytes;
  static constexpr int kScaleDmas = kNT / 2;
  static constexpr int kSlot = kTiles + (kRows + kCols) * 4;
  static constexpr int kSlots = kNT == 2 ? 4 : 3;
  static constexpr int kDmas = 4 + 2 * kNT + kScaleDmas;
};

typedef float v16_t __attribute__((ext_vector_type(16)));

// One block of K: codes of a 32-row tile, chunks h, 2 + h, 4 + h, 6 + h of the
// lane's row; and all of a wave's, with their scales.
struct Frag {
  u32x4_t c[4];
};
template <int kNT>
struct Frags {
  Frag a[2], b[kNT];
  uint32_t sa[2], sb[kNT];
};

template <Fp8Type kA>
__device__ __forceinline__ v16_t mfma_fp8_32(const Frag& x, const Frag& y, int s, v16_t c,
                                             uint32_t sx, uint32_t sy) {
  const u32x4_t x0 = x.c[2 * s], x1 = x.c[2 * s + 1], y0 = y.c[2 * s], y1 = y.c[2 * s + 1];
  const v8i_t xv = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3],
                    (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  const v8i_t yv = {(int)y0[0], (int)y0[1], (int)y0[2], (int)y0[3],
                    (int)y1[0], (int)y1[1], (int)y1[2], (int)y1[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xv, yv, c, kE4M3, kA, 0, (int)sx, 0,
                                                         (int)sy);
}

// Pieces that a step's products come in, each with a share of the next step's
// reads and of the DMAs beside it.
template <int kNT, bool kBf16>
constexpr int kPiecesOf = kBf16 ? 8 : 2 * kNT;
template <int n>
using Int = std::integral_constant<int, n>;
template <class F, int... n>
__device__ __forceinline__ void for_each(F f, std::integer_sequence<int, n...>) {
  (f(Int<n>()), ...);
}

// acc += the products of one step; beside(Int<n>) goes out with piece n. Without
// that order, kept by fences, the compiler moved the reads behind the matrix
// instructions and then waited for them (512 x 8192 x 8192 47 us).
template <bool kBf16, bool kF32Scale, Fp8Type kA, int kNT, class Beside>
__device__ __forceinline__ void multiply(v16_t (&acc)[2][kNT], const Frags<kNT>& f,
                                         Beside beside) {
  const auto pieces = std::make_integer_sequence<int, kPiecesOf<kNT, kBf16>>();
  if constexpr (kBf16) {
    v16_t sums[2][kNT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kNT; ++j) sums[i][j] = kF32Scale ? v16_t{} : acc[i][j];
    for_each([&](auto n) {
      constexpr int c = n() / 2, e = n() % 2;
      bf16x8_t a[2], b[kNT];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[i] = fp8x8_to_bf16<kA>(f.a[i].c[c][2 * e], f.a[i].c[c][2 * e + 1],
                                 kF32Scale ? 1.0f : fp8_scale_value(f.sa[i]));
#pragma unroll
      for (int j = 0; j < kNT; ++j)
        b[j] = fp8x8_to_bf16<kE4M3>(f.b[j].c[c][2 * e], f.b[j].c[c][2 * e + 1],
                                    kF32Scale ? 1.0f : fp8_scale_value(f.sb[j]));
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          sums[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], sums[i][j], 0, 0, 0);
      beside(n);
      __builtin_amdgcn_sched_barrier(0);
    }, pieces);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        if constexpr (kF32Scale) {
          const float scale = __uint_as_float(f.sa[i]) * __uint_as_float(f.sb[j]);
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(scale, sums[i][j][v], acc[i][j][v]);
        } else {
          acc[i][j] = sums[i][j];
        }
      }
  } else if constexpr (kF32Scale) {
    // A tile's sums are added while the next one's are made.
    v16_t sums[2];
    const auto add = [&](int t) {
      const float scale = __uint_as_float(f.sa[t / kNT]) * __uint_as_float(f.sb[t % kNT]);
      v16_t& to = acc[t / kNT][t % kNT];
#pragma unroll
      for (int v = 0; v < 16; ++v) to[v] = fmaf(scale, sums[t & 1][v], to[v]);
    };
    for_each([&](auto n) {
      constexpr int i = n() / kNT, j = n() % kNT;
      v16_t d = mfma_fp8_32<kA>(f.b[j], f.a[i], 0, v16_t{}, 127, 127);
      sums[n() & 1] = mfma_fp8_32<kA>(f.b[j], f.a[i], 1, d, 127, 127);
      if constexpr (n() > 0) add(n() - 1);
      beside(n);
      __builtin_amdgcn_sched_barrier(0);
    }, pieces);
    add(2 * kNT - 1);
  } else {
    for_each([&](auto n) {
      constexpr int i = n() / kNT, j = n() % kNT;
      acc[i][j] = mfma_fp8_32<kA>(f.b[j], f.a[i], 0, acc[i][j], f.sb[j], f.sa[i]);
      acc[i][j] = mfma_fp8_32<kA>(f.b[j], f.a[i], 1, acc[i][j], f.sb[j], f.sa[i]);
      beside(n);
      __builtin_amdgcn_sched_barrier(0);
    }, pieces);
  }
}

// A byte per lane, into the lane's dword of LDS.
__device__ __forceinline__ void dma1(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, off"
               :: "v"(g), "s"(lds) : "m0");
}

template <int kLeft>
__device__ __forceinline__ void wait_loads_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(kLeft) : "memory");
}

template <int kNT, bool kBf16, bool kF32Scale, Fp8Out kOut, Fp8Type kA, bool kTail>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_kernel(Fp8GemmArgs p, int tiles_m, int tiles_n) {
  constexpr bool kGlu = kOut == kFp8Glu;
  using G = Geom<kNT>;
  __shared__ __align__(16) uint8_t lds[G::kSlots * G::kSlot];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wy = wave >> 1, wx = wave & 1;
  const int r = lane & 31, h = lane >> 5;
  const int id = workgroup_id(tiles_m * tiles_n);
  if (id < 0) return;
  int tm, tn;
  xcd_tile(id, tiles_m, tiles_n, kGroupM, tm, tn);
  const int row0 = tm * kRows;
  const int col0 = tn * (kGlu ? G::kCols / 2 : G::kCols);

  // B's row of tile row t. kGlu: a tile is 64 columns of act, wave column wx has
  // 32 of them, its first tile their gate rows, its second their up rows.
  static_assert(!kGlu || kNT == 2);
  const auto b_row = [&](int t) -> int64_t {
    if constexpr (kGlu)
      return (int64_t)min(col0 + 32 * (t >> 6) + (t & 31), p.N - 1) + ((t >> 5) & 1) * (int64_t)p.N;
    else
      return min(col0 + t, p.N - 1);
  };

  // This wave's DMAs: tile rows 32 w + 8 q + lane / 8 of A, 16 kNT w + 8 q + lane
  // / 8 of B; lane l lands at chunk l % 8 of its row and so fetches chunk (l % 8)
  // ^ swizzle.
  const uint8_t* from_a[4];
  const uint8_t* from_b[2 * kNT];
  int chunk[2];
#pragma unroll
  for (int q = 0; q < 2 * kNT; ++q) {
    const int t = 8 * q + (lane >> 3);
    const int c = (lane & 7) ^ chunk_swizzle(t);  // the swizzle repeats every 16 rows
    if (q < 2) chunk[q] = c;
    if (q < 4)
      from_a[q < 4 ? q : 0] = p.A + (int64_t)min(row0 + 32 * wave + t, p.M - 1) * p.K + 16 * c;
    from_b[q] = p.B + b_row(16 * kNT * wave + t) * p.K + 16 * c;
  }
  // Scales: piece n of 64 rows, A's two and then B's.
  const uint8_t* from_s[G::kScaleDmas];
  int piece[G::kScaleDmas];
#pragma unroll
  for (int e = 0; e < G::kScaleDmas; ++e) {
    int n = wave + 4 * e;
    if (n >= 2 + kNT) n -= 2;  // two waves repeat the last two, the same bytes
    piece[e] = n;
    const int64_t at =
        n < 2 ? (int64_t)min(row0 + 64 * n + lane, p.M - 1) * p.kblocks
              : (b_row(64 * (n - 2) + lane) >> p.b_shift) * p.kblocks;
    from_s[e] = static_cast<const uint8_t*>(n < 2 ? p.As : p.Bs) + (kF32Scale ? 4 : 1) * at;
  }
  const uint32_t lds0 = lds_addr(lds);
  const int last = p.kblocks - 1;
  const int last_bytes = p.K - last * kFp8Block;
  // DMA n of a step: A's four, B's 2 kNT, the scales'.
  const auto load = [&](auto n, int k, uint32_t slot) {
    constexpr int q = n() < 4 ? n() : n() - 4;
    if constexpr (q < 2 * kNT) {
      const int64_t at = (int64_t)k * kRowBytes;
      const uint8_t* g = (n() < 4 ? from_a[q < 4 ? q : 0] : from_b[q]) + at;
      if (kTail) g = 16 * chunk[q & 1] < (k == last ? last_bytes : kRowBytes) ? g : kFp8Zeros;
      const uint32_t to = n() < 4 ? wave * 4096 : kRows * kRowBytes + wave * 2048 * kNT;
      dma16(g, __builtin_amdgcn_readfirstlane(lds0 + slot + to) + 1024 * q);
    } else {
      constexpr int e = q - 2 * kNT;
      const uint32_t to =
          __builtin_amdgcn_readfirstlane(lds0 + slot + G::kTiles + 256 * piece[e]);
      if constexpr (kF32Scale)
        dma4(from_s[e] + (int64_t)4 * k, to);
      else
        dma1(from_s[e] + k, to);
    }
  };
  const auto load_step = [&](int kb, uint32_t slot) {
    for_each([&](auto n) { load(n, min(kb, last), slot); },
             std::make_integer_sequence<int, G::kDmas>());
  };

  const uint32_t x = (uint32_t)(h ^ chunk_swizzle(r));
  const uint32_t frag_a = (uint32_t)(64 * wy + r) * kRowBytes;
  const uint32_t frag_b = (uint32_t)(kRows + 32 * kNT * wx + r) * kRowBytes;
  uint32_t at_a[4], at_b[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    at_a[c] = frag_a + 16 * ((2 * c) ^ x);
    at_b[c] = frag_b + 16 * ((2 * c) ^ x);
  }
  // Read n of a step: scales, then the four chunks of B's tiles and of A's.
  constexpr int kReads = 5 * (2 + kNT);
  const auto read = [&](auto n, uint32_t slot, Frags<kNT>& f) {
    const uint8_t* base = lds + slot;
    if constexpr (n() < 2 + kNT) {
      const uint32_t* s = reinterpret_cast<const uint32_t*>(base + G::kTiles);
      if constexpr (n() < 2)
        f.sa[n()] = s[64 * wy + 32 * n() + r];
      else
        f.sb[n() - 2] = s[kRows + 32 * kNT * wx + 32 * (n() - 2) + r];
    } else {
      constexpr int t = (n() - 2 - kNT) % (2 + kNT), c = (n() - 2 - kNT) / (2 + kNT);
      if constexpr (t < kNT)
        f.b[t].c[c] = *reinterpret_cast<const u32x4_t*>(base + at_b[c] + t * 32 * kRowBytes);
      else
        f.a[t - kNT].c[c] =
            *reinterpret_cast<const u32x4_t*>(base + at_a[c] + (t - kNT) * 32 * kRowBytes);
    }
  };

  v16_t acc[2][kNT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < kNT; ++j) acc[i][j] = v16_t{};

  for (int s = 0; s < G::kSlots; ++s) load_step(s, s * G::kSlot);
  wait_loads_and_meet<G::kDmas*(G::kSlots - 1)>();
  uint32_t now = 0, next = G::kSlot;  // slots of steps kb and kb + 1
  const auto step = [&](int kb, Frags<kNT>& f, Frags<kNT>& g) {
    // Step kb + 1 has landed, in all waves, and step kb is in their registers.
    wait_loads_and_meet<G::kDmas*(G::kSlots - 2)>();
    const int k = min(kb + G::kSlots, last);  // past the last it is loaded again, and not used
    multiply<kBf16, kF32Scale, kA, kNT>(acc, f, [&](auto n) {
      constexpr int kPieces = kPiecesOf<kNT, kBf16>;
      // The reads leave out the last piece, so that they have returned at the end.
      constexpr int r0 = kReads * n() / (kPieces - 1), r1 = kReads * (n() + 1) / (kPieces - 1);
      constexpr int d0 = G::kDmas * n() / kPieces, d1 = G::kDmas * (n() + 1) / kPieces;
      if constexpr (n() < kPieces - 1)
        for_each([&](auto m) { read(Int<r0 + m()>(), next, g); },
                 std::make_integer_sequence<int, r1 - r0>());
      for_each([&](auto m) { load(Int<d0 + m()>(), k, now); },
               std::make_integer_sequence<int, d1 - d0>());
    });
    now = next;
    next = next + G::kSlot == G::kSlots * G::kSlot ? 0 : next + G::kSlot;
  };
  Frags<kNT> f, g;
  for_each([&](auto n) { read(n, 0, f); }, std::make_integer_sequence<int, kReads>());
  int kb = 0;
  for (; kb + 2 <= p.kblocks; kb += 2) {
    step(kb, f, g);
    step(kb + 1, g, f);
  }
  if (kb < p.kblocks) step(kb, f, g);
  wait_loads_and_meet<0>();

  // Register 4 q + t of tile (i, j) holds row 32 i + r, column 32 j + 8 q + 4 h
  // + t of the wave's part. Each wave parks it in its own 16 KiB and stores
  // whole lines: FP32 rows of 64 columns as 256 bytes, 16-byte chunk c at c ^
  // (row % 16); BF16 rows of `width` columns as 128 bytes, chunk c at c ^ (row
  // % 8).
  uint8_t* park = lds + wave * 16384;
  const int m_wave = row0 + 64 * wy;
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
  } else {
#pragma unroll
    for (int part = 0; part < kNT / 2; ++part) {
      const int ncol = col0 + 32 * kNT * wx + 64 * part, cols = p.N - ncol;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v16_t& v = acc[i][2 * part + j];
            const int c = 8 * j + 2 * q + h, row = 32 * i + r;
            if constexpr (kOut == kFp8Bf16)
              park_bf16(row, 4 * c, pack_bf16x2(v[4 * q], v[4 * q + 1]),
                        pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
            else
              *reinterpret_cast<float4*>(park + row * 256 + 16 * (c ^ (row & 15))) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
      if constexpr (kOut == kFp8Bf16) {
        store_bf16(static_cast<uint16_t*>(p.C) + (int64_t)m_wave * p.N + ncol, p.N, cols, 64);
      } else {
        float* to = static_cast<float*>(p.C) + (int64_t)m_wave * p.N + ncol;
        if (p.N % 4 == 0) {
          for (int x0 = 0; x0 < 64; x0 += 4) {
            const int row = x0 + (lane >> 4), c = lane & 15;
            const float4 v =
                *reinterpret_cast<const float4*>(park + row * 256 + 16 * (c ^ (row & 15)));
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
  }
}

template <int kNT, bool kBf16, bool kF32Scale, Fp8Out kOut, Fp8Type kA>
hipError_t launch(const Fp8GemmArgs& a, hipStream_t stream) {
  constexpr int kCols = kOut == kFp8Glu ? Geom<kNT>::kCols / 2 : Geom<kNT>::kCols;
  const int64_t tiles_m = ((int64_t)a.M + kRows - 1) / kRows;
  const int64_t tiles_n = ((int64_t)a.N + kCols - 1) / kCols;
  const dim3 grid = grid_of(tiles_m * tiles_n, kThreads);
  if (a.K % kFp8Block != 0)
    hipLaunchKernelGGL((gemm_fp8_kernel<kNT, kBf16, kF32Scale, kOut, kA, true>), grid,
                       dim3(kThreads), 0, stream, a, (int)tiles_m, (int)tiles_n);
  else
    hipLaunchKernelGGL((gemm_fp8_kernel<kNT, kBf16, kF32Scale, kOut, kA, false>), grid,
                       dim3(kThreads), 0, stream, a, (int)tiles_m, (int)tiles_n);
  return hipGetLastError();
}

template <bool kBf16, bool kF32Scale, Fp8Out kOut, Fp8Type kA>
hipError_t launch_sized(const Fp8GemmArgs& a, hipStream_t stream) {
  // Wide tiles read less of A and B for a product, where they still fill the chip
  // (FP32 scales: 16384 x 4096 x 14336 1145 against 1331 us, 2048 x 4096 x 4096, 256
  // of them, 47 against 55; 2048 x 2048 x 2048, half of that, 23.6 against 15.6).
  const int64_t wide = ((int64_t)a.M + 127) / 128 * (((int64_t)a.N + 255) / 256);
  if constexpr (kBf16 && kF32Scale)  // the registers do not do for 128 x 256
    return launch<2, kBf16, kF32Scale, kOut, kA>(a, stream);
  else
    return wide >= 256 ? launch<4, kBf16, kF32Scale, kOut, kA>(a, stream)
                     : launch<2, kBf16, kF32Scale, kOut, kA>(a, stream);
}

template <Fp8Type kA>
hipError_t launch_typed(const Fp8GemmArgs& a, Fp8Out out, bool f32, hipStream_t stream) {
  if (out == kFp8F32)
    return f32 ? launch_sized<true, true, kFp8F32, kA>(a, stream)
               : launch_sized<true, false, kFp8F32, kA>(a, stream);
  return f32 ? launch_sized<false, true, kFp8Bf16, kA>(a, stream)
             : launch<2, false, false, kFp8Bf16, kA>(a, stream);
}

int64_t tiles(int64_t M, int64_t N, int64_t side) {
  return (M + side - 1) / side * ((N + side - 1) / side);
}

// Whether a product goes to the kernel that splits K over its waves: few rows; few
// tiles of a long K (128 x 8192 x 4096 16.8 us there, 128 x 4096 x 4096 10.6 against
// 15.2 here; but 128 x 28672 x 4096 58 against 34); or at most 512 tiles of 32 x 16, two
// a CU, whatever K (128 x 2048 x 2048 7.4 us there, 9.3 here, FP32 results 7.2 and
// 15.2; 512 x 512 x 512 5.0 and 5.3, x 1024 6.9 and 6.6; but 512 x 2048 x 2048, past
// that, 11.9 against 9.5).
bool few_tiles(int64_t M, int64_t N, int64_t kblocks) {
  return M <= 64 || (M + 31) / 32 * ((N + 15) / 16) <= 512 ||
         (tiles(M, N, 128) <= 64 && kblocks >= 32);
}
// 256 x 256 tiles where they fill half the chip, which is two rounds of tiles
// here (1024 x 8192 x 8192 82 against 91 us; 1024 x 4096 x 4096 41 against 19).
bool big_tiles(int64_t M, int64_t N) { return M > 64 && tiles(M, N, 256) >= 128; }

}  // namespace

hipError_t launch_gemm_fp8(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type, bool scale_f32,
                           hipStream_t stream) {
  if (few_tiles(a.M, a.N, a.kblocks) ||
      (!scale_f32 && fp8_short_scales(a.M, a.N, a.kblocks, a.b_shift)))
    return launch_gemm_fp8_small(a, out, a_type, scale_f32, stream);
  if (out == kFp8Bf16 && !scale_f32 && big_tiles(a.M, a.N))
    return launch_gemm_fp8_tile(a, out, a_type, Fp8ActOut{}, stream);
  return a_type == kE4M3 ? launch_typed<kE4M3>(a, out, scale_f32, stream)
                         : launch_typed<kE5M2>(a, out, scale_f32, stream);
}

bool gemm_fp8_swiglu_small(int64_t M, int64_t I, int64_t K) {
  // The large tiles' offsets from gate's rows to up's have 32 bits.
  return !big_tiles(M, 2 * I) || (I + 128) * K >= (int64_t(1) << 32) - 4096 ||
         fp8_short_scales(M, 2 * I, (K + kFp8Block - 1) / kFp8Block, 7);
}

hipError_t launch_gemm_fp8_swiglu(const Fp8GemmArgs& a, uint8_t* codes, uint8_t* scales,
                                  void* workspace, hipStream_t stream) {
  if (!gemm_fp8_swiglu_small(a.M, a.N, a.K))
    return launch_gemm_fp8_tile(a, kFp8Glu, kE4M3, Fp8ActOut{codes, scales}, stream);
  Fp8GemmArgs g = a;
  if (!g.C) g.C = workspace;
  const int64_t rows = 2 * (int64_t)a.N;
  const hipError_t e = few_tiles(a.M, rows, a.kblocks) || fp8_short_scales(a.M, rows, a.kblocks, 7)
                           ? launch_gemm_fp8_small(g, kFp8Glu, kE4M3, false, stream)
                           : launch<2, false, false, kFp8Glu, kE4M3>(g, stream);
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
