// FP8 GEMM of UE8M0-scaled operands on 256 x 256 tiles, for many rows: C in
// BF16, or the gate+up product of a gated MLP whose activation is quantized in
// the epilogue (kFp8Glu). The FP8 matrix instructions bound it: 2 M N K
// operations at v_mfma_scale_f32_32x32x64_f8f6f4's 64 cycles an instruction.
//
// Tiling. One workgroup of 4 waves (one per SIMD) owns a 256 x 256 tile, wave
// (wy, wx) a 128 x 128 part: 4 x 4 tiles of 32 x 32, whose 256 accumulators a
// lane live in the accumulation registers. B's fragment is the first operand,
// so a lane ends with four consecutive columns of one row of C. UE8M0 scales go
// into the instruction: a block of 128 has one byte a row of A, and one a wave
// (B in 128 x 128 blocks) or a row of B.
//
// Data movement. A K step is one block of 128: 128 bytes a row, a whole line,
// two slices of 64 for the instruction. Tiles go global -> LDS by DMA (8 rows an
// instruction, addresses from a wave-uniform base and per-lane offsets prepared
// once) into two slots of A and three of B (160 KiB), in rows of eight 16-byte
// chunks XOR-swizzled by the row, so that fragment reads fall on all banks.
//
// Schedule of a step. The fragments of a slice have two sets of registers: the 16
// reads of the next slice go out beside the first instructions of this one, a
// slice ahead of their use (with one set, read behind the last use, a fifth of
// the time went into waiting for LDS reads). Between the two slices of a step
// the waves meet: the step has been read, the next one's tiles have landed, and
// the DMAs of the step after next go out beside the instructions, A's a whole
// step ahead, B's, which have a third slot, one and a half.
//
// Measured: 8192^3 395 us (2.78 PFLOP/s; 128 x 128 tiles 643, one set of fragments
// and two slots 425, three slots of B 397 before the K rotation below), 16384 x
// 4096 x 14336 675, gate+up 16384 x 4096 x 14336 with g and u 1582. The
// instructions alone run at 3.67 PFLOP/s, where power ends them; the tiles come
// from L2 at 11 TB/s, which neither more DMAs under way nor other orders moved.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "fp8.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 256;
constexpr int kRowBytes = kFp8Block;
constexpr int kSlot = kTile * kRowBytes;  // 32 KiB: one operand's K step
constexpr int kGroupM = 4;
constexpr uint32_t kBias = 3 * 1024;      // keeps per-lane offsets positive, see dma_pair

// What a lane needs to move and read one tile.
struct Ctx {
  uint32_t off_a[8], off_b[8];  // DMA q's per-lane offset from base_a, base_b
  const uint8_t* base_a;        // wave-uniform, less kBias
  const uint8_t* base_b;
  uint32_t lds;                 // of this wave's rows in slot 0 of A
  uint32_t fa[4], fb[4];        // fragment reads of quarter q of a step, slot 0
  int last;                     // last K step
  int rot;                      // the K step this tile begins with
  int tail_bytes;               // of the last step, where K % 128 != 0
  int chunk[2];                 // the chunk a lane fetches, rows at 0 and 8 mod 16
};

// DMAs Q0, Q0 + 1 of an operand: 8 tile rows each. The instruction's immediate
// moves the global and the LDS address alike, so one M0 serves four DMAs, and
// the per-lane offsets have the immediate taken off and kBias added.
template <int Q0>
__device__ __forceinline__ void dma_pair(const uint8_t* base, uint32_t off0, uint32_t off1,
                                         uint32_t m0) {
  asm volatile(
      "s_mov_b32 m0, %3\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %2 offset:%4\n\t"
      "global_load_lds_dwordx4 %1, %2 offset:%5"
      :: "v"(off0), "v"(off1), "s"(sgpr_ptr(base)), "s"(m0), "n"((Q0 % 4) * 1024),
         "n"(((Q0 + 1) % 4) * 1024)
      : "m0");
}

// kOp: 0 = A, 1 = B. A last step that ends inside a block takes its chunks past
// K from a line of zeros.
template <int kOp, int Q0, bool kTail>
__device__ __forceinline__ void load_pair(const Ctx& c, int kb, uint32_t slot) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(c.lds + slot + (Q0 / 4) * 4096);
  const uint8_t* base = (kOp ? c.base_b : c.base_a) + (int64_t)kb * kRowBytes;
  const uint32_t o0 = kOp ? c.off_b[Q0] : c.off_a[Q0];
  const uint32_t o1 = kOp ? c.off_b[Q0 + 1] : c.off_a[Q0 + 1];
  if constexpr (kTail) {
    // Without a branch: one in the K loop lets the compiler move the matrix
    // instructions out of their places, into the next basic block.
    const uint8_t* g0 = base + o0 + (Q0 % 4) * 1024;
    const uint8_t* g1 = base + o1 + ((Q0 + 1) % 4) * 1024;
    const int bytes = kb == c.last ? c.tail_bytes : kRowBytes;
    g0 = 16 * c.chunk[0] < bytes ? g0 : kFp8Zeros;
    g1 = 16 * c.chunk[1] < bytes ? g1 : kFp8Zeros;
    dma16(g0, m0 + (Q0 % 4) * 1024);
    dma16(g1, m0 + ((Q0 + 1) % 4) * 1024);
  } else {
    dma_pair<Q0>(base, o0, o1, m0);
  }
}

// The K step loaded as step t (a tile's steps go around from rot); past the
// last it is loaded again, and not used.
__device__ __forceinline__ int phys_step(const Ctx& c, int t) {
  const int k = min(t, c.last) + c.rot;
  return k > c.last ? k - c.last - 1 : k;
}

// 32 codes of one row, half a 64-wide slice of K; and a wave's fragments of one
// slice.
struct Frag {
  u32x4_t half[2];
};
struct Frags {
  Frag a[4], b[4];
};

// Read kRead (0 .. 15) of the fragments of a slice: B's eight halves, then A's.
template <int kSlice, int kRead>
__device__ __forceinline__ void read_half(const Ctx& c, const uint8_t* lds_a, const uint8_t* lds_b,
                                          Frags& f) {
  constexpr int kTileOf = (kRead & 7) >> 1, kHalf = kRead & 1;
  const uint8_t* p = (kRead < 8 ? lds_b + c.fb[2 * kSlice + kHalf]
                                : lds_a + c.fa[2 * kSlice + kHalf]) + kTileOf * 32 * kRowBytes;
  (kRead < 8 ? f.b[kTileOf] : f.a[kTileOf]).half[kHalf] = *reinterpret_cast<const u32x4_t*>(p);
}

template <int... kReads>
__device__ __forceinline__ void read_all(const Ctx& c, const uint8_t* lds_a, const uint8_t* lds_b,
                                         Frags& f, std::integer_sequence<int, kReads...>) {
  (read_half<0, kReads>(c, lds_a, lds_b, f), ...);
}

template <Fp8Type kA>
__device__ __forceinline__ void mma(v16f_t& acc, const Frag& x, const Frag& y, uint32_t sx,
                                    uint32_t sy) {
  const u32x4_t x0 = x.half[0], x1 = x.half[1], y0 = y.half[0], y1 = y.half[1];
  const v8i_t xv = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3],
                    (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
  const v8i_t yv = {(int)y0[0], (int)y0[1], (int)y0[2], (int)y0[3],
                    (int)y1[0], (int)y1[1], (int)y1[2], (int)y1[3]};
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xv, yv, acc, kE4M3, kA, 0, (int)sx, 0,
                                                        (int)sy);
}

#define MXFP4_FENCE() __builtin_amdgcn_sched_barrier(0)

// End of a group of two matrix instructions: so many LDS reads after the first
// and after the second.
template <int kFirst, int kSecond>
__device__ __forceinline__ void group_end() {
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  if constexpr (kFirst > 0) __builtin_amdgcn_sched_group_barrier(0x100, kFirst, 0);
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  if constexpr (kSecond > 0) __builtin_amdgcn_sched_group_barrier(0x100, kSecond, 0);
  MXFP4_FENCE();
}

// Scale words: bytes of four K steps of the rows of A's tiles, and of B's (kNB:
// one, gate's and up's, or each tile's).
template <int kNB>
struct Scales {
  uint32_t a[4], b[kNB];
};

template <int kNB>
struct ScaleRows {
  const uint8_t* As;
  const uint8_t* Bs;
  int64_t a[4], b[kNB], a_total, b_total;
};

template <int kNB>
__device__ __forceinline__ void load_scales(const ScaleRows<kNB>& w, int kb, Scales<kNB>& s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s.a[i] = scale_word(w.As, w.a[i] + kb, w.a_total);
#pragma unroll
  for (int j = 0; j < kNB; ++j) s.b[j] = scale_word(w.Bs, w.b[j] + kb, w.b_total);
}

// Offsets of B's three slots: of steps T, T + 1 and T + 2.
struct Ring {
  uint32_t now, next, free;
};

// The 16 matrix instructions of one slice on fragments f, with the 16 reads of
// the next slice (kSlice of the step in lds_a, lds_b) into g and the four pairs
// of DMAs of operand kOp for step k into `slot`. The reads come early, so that
// they have returned when the slice ends.
template <Fp8Type kA, int kNB, bool kTail, int kSlice, int kOp>
__device__ __forceinline__ void slice(const Ctx& c, v16f_t (&acc)[4][4], const Frags& f, Frags& g,
                                      const uint8_t* lds_a, const uint8_t* lds_b,
                                      const Scales<kNB>& s, int k, uint32_t slot) {
  const auto sb = [&](int j) { return s.b[kNB == 1 ? 0 : kNB == 2 ? j & 1 : j]; };
#define MXFP4_MMA2(i, j)                                           \
  mma<kA>(acc[i][j], f.b[j], f.a[i], sb(j), s.a[i]);               \
  mma<kA>(acc[i][(j) + 1], f.b[(j) + 1], f.a[i], sb((j) + 1), s.a[i])
#define MXFP4_READ(n) read_half<kSlice, n>(c, lds_a, lds_b, g)
  MXFP4_MMA2(0, 0);
  MXFP4_READ(0);
  MXFP4_READ(1);
  MXFP4_READ(2);
  load_pair<kOp, 0, kTail>(c, k, slot);
  group_end<2, 1>();
  MXFP4_MMA2(0, 2);
  MXFP4_READ(3);
  MXFP4_READ(4);
  MXFP4_READ(5);
  group_end<2, 1>();
  MXFP4_MMA2(1, 0);
  MXFP4_READ(6);
  MXFP4_READ(7);
  MXFP4_READ(8);
  load_pair<kOp, 2, kTail>(c, k, slot);
  group_end<2, 1>();
  MXFP4_MMA2(1, 2);
  MXFP4_READ(9);
  MXFP4_READ(10);
  MXFP4_READ(11);
  group_end<2, 1>();
  MXFP4_MMA2(2, 0);
  MXFP4_READ(12);
  MXFP4_READ(13);
  load_pair<kOp, 4, kTail>(c, k, slot);
  group_end<1, 1>();
  MXFP4_MMA2(2, 2);
  MXFP4_READ(14);
  MXFP4_READ(15);
  group_end<1, 1>();
  MXFP4_MMA2(3, 0);
  load_pair<kOp, 6, kTail>(c, k, slot);
  group_end<0, 0>();
  MXFP4_MMA2(3, 2);
  group_end<0, 0>();
#undef MXFP4_MMA2
#undef MXFP4_READ
}

// One K step T, P = T % 4, A in slot P % 2: f holds its first slice.
template <Fp8Type kA, int kNB, bool kTail, int P>
__device__ __forceinline__ void k_step(const Ctx& c, const uint8_t* lds, v16f_t (&acc)[4][4],
                                       Frags& f, Frags& g, const ScaleRows<kNB>& rows,
                                       Scales<kNB>& s, Scales<kNB>& next, Ring& ring, int T) {
  constexpr uint32_t kSlotA = (P & 1) * kSlot;
  const int k2 = phys_step(c, T + 2);
  slice<kA, kNB, kTail, 1, 1>(c, acc, f, g, lds + kSlotA, lds + ring.now, s, k2, ring.free);
  // All but the last 8 loads (step T + 2's B): step T + 1 has landed; and this
  // step has been read.
  asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  MXFP4_FENCE();
  if constexpr (P == 3) {
    // The next words were loaded two steps before: landed by now.
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(next.a[i]));
#pragma unroll
    for (int j = 0; j < kNB; ++j) asm volatile("" : "+v"(next.b[j]));
  }
  if constexpr (P == 1) load_scales(rows, phys_step(c, T + 3), next);
  slice<kA, kNB, kTail, 0, 0>(c, acc, g, f, lds + (kSlot - kSlotA), lds + ring.next, s, k2, kSlotA);
  ring = Ring{ring.next, ring.free, ring.now};
  if constexpr (P == 3) {
    s = next;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) s.a[i] >>= 8;
#pragma unroll
    for (int j = 0; j < kNB; ++j) s.b[j] >>= 8;
  }
}

template <Fp8Out kOut, Fp8Type kA, bool kRowsB, bool kTail>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_fp8_tile_kernel(Fp8GemmArgs p, int tiles_m, int tiles_n, Fp8ActOut act) {
  constexpr bool kGlu = kOut == kFp8Glu;
  constexpr int kNB = kRowsB ? 4 : kGlu ? 2 : 1;
  __shared__ __align__(16) uint8_t lds[5 * kSlot];  // A's slots 0, 1, then B's 0, 1, 2

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

  // B's row of tile row t. kGlu: a tile is 128 columns of act; tile row 128 wx +
  // 32 j + rr is the gate (j even) or up (j odd) row of column 64 wx + 32 (j / 2)
  // + rr, so that a wave holds both of its 64 columns.
  const auto b_row = [&](int t) -> int64_t {
    if constexpr (kGlu)
      return (int64_t)(col0 + 64 * (t >> 7) + 32 * ((t >> 6) & 1) + (t & 31)) +
             ((t >> 5) & 1) * (int64_t)p.N;
    else
      return min(col0 + t, p.N - 1);
  };

  Ctx c;
  c.last = p.kblocks - 1;
  // XCD x starts x / 8 into K, and every other tile of its neighbourhood 4 steps
  // further on, so that the tiles that share rows of an operand do not all wait
  // for the same lines (16384 x 28672 x 4096 1475 -> 1456 us). Where the scales
  // of K are not whole words, steps begin at 0.
  c.rot = kTail || p.kblocks % 4 != 0
              ? 0
              : (4 * ((id % 8) * (p.kblocks / 4) / 8) + 4 * ((tm + tn) & 1)) % p.kblocks;
  c.tail_bytes = p.K - c.last * kFp8Block;
  c.lds = lds_addr(lds) + wave * 8192;
  const int64_t a_first = min(row0 + 64 * wave, p.M - 1);
  const int64_t b_first = b_row(64 * wave);
  c.base_a = p.A + a_first * p.K - kBias;
  c.base_b = p.B + b_first * p.K - kBias;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int t = 64 * wave + 8 * q + (lane >> 3);
    const int chunk = (lane & 7) ^ chunk_swizzle(t);
    if (q < 2) c.chunk[q] = chunk;
    const uint32_t from = 16 * chunk + kBias - (q % 4) * 1024;
    c.off_a[q] = (uint32_t)(min(row0 + t, p.M - 1) - (int)a_first) * (uint32_t)p.K + from;
    // Up's rows lie I rows behind gate's: within 32 bits (gemm_fp8_swiglu_small).
    c.off_b[q] = (uint32_t)(b_row(t) - b_first) * (uint32_t)p.K + from;
  }
  const uint32_t x = (uint32_t)(h ^ chunk_swizzle(r)) << 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    c.fa[q] = (uint32_t)(128 * wy + r) * kRowBytes + ((32u * q) ^ x);
    c.fb[q] = (uint32_t)(128 * wx + r) * kRowBytes + ((32u * q) ^ x);
  }

  ScaleRows<kNB> rows;
  rows.As = static_cast<const uint8_t*>(p.As);
  rows.Bs = static_cast<const uint8_t*>(p.Bs);
  rows.a_total = (int64_t)p.M * p.kblocks;
  const int64_t b_rows = kGlu ? 2 * (int64_t)p.N : p.N;
  rows.b_total = ((b_rows + (1 << p.b_shift) - 1) >> p.b_shift) * p.kblocks;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    rows.a[i] = (int64_t)min(row0 + 128 * wy + 32 * i + r, p.M - 1) * p.kblocks;
#pragma unroll
  for (int j = 0; j < kNB; ++j)
    rows.b[j] = (b_row(128 * wx + 32 * j + (kRowsB ? r : 0)) >> p.b_shift) * p.kblocks;

  Scales<kNB> s, next;
  load_scales(rows, c.rot, s);
  next = s;
  Ring ring{2 * kSlot, 3 * kSlot, 4 * kSlot};
  const int k0 = c.rot, k1 = phys_step(c, 1);
  load_pair<0, 0, kTail>(c, k0, 0);
  load_pair<0, 2, kTail>(c, k0, 0);
  load_pair<0, 4, kTail>(c, k0, 0);
  load_pair<0, 6, kTail>(c, k0, 0);
  load_pair<1, 0, kTail>(c, k0, ring.now);
  load_pair<1, 2, kTail>(c, k0, ring.now);
  load_pair<1, 4, kTail>(c, k0, ring.now);
  load_pair<1, 6, kTail>(c, k0, ring.now);
  load_pair<1, 0, kTail>(c, k1, ring.next);
  load_pair<1, 2, kTail>(c, k1, ring.next);
  load_pair<1, 4, kTail>(c, k1, ring.next);
  load_pair<1, 6, kTail>(c, k1, ring.next);
  load_pair<0, 0, kTail>(c, k1, kSlot);
  load_pair<0, 2, kTail>(c, k1, kSlot);
  load_pair<0, 4, kTail>(c, k1, kSlot);
  load_pair<0, 6, kTail>(c, k1, kSlot);
  v16f_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v16f_t{};
  // Step 0 has landed; the 16 DMAs of step 1 may be under way.
  asm volatile("s_waitcnt vmcnt(16)\n\ts_barrier" ::: "memory");
  Frags f, g;
  read_all(c, lds, lds + ring.now, f, std::make_integer_sequence<int, 16>());
  int T = 0;
  for (; T + 4 <= p.kblocks; T += 4) {
    k_step<kA, kNB, kTail, 0>(c, lds, acc, f, g, rows, s, next, ring, T);
    k_step<kA, kNB, kTail, 1>(c, lds, acc, f, g, rows, s, next, ring, T + 1);
    k_step<kA, kNB, kTail, 2>(c, lds, acc, f, g, rows, s, next, ring, T + 2);
    k_step<kA, kNB, kTail, 3>(c, lds, acc, f, g, rows, s, next, ring, T + 3);
  }
  if (T < p.kblocks) k_step<kA, kNB, kTail, 0>(c, lds, acc, f, g, rows, s, next, ring, T);
  if (T + 1 < p.kblocks) k_step<kA, kNB, kTail, 1>(c, lds, acc, f, g, rows, s, next, ring, T + 1);
  if (T + 2 < p.kblocks) k_step<kA, kNB, kTail, 2>(c, lds, acc, f, g, rows, s, next, ring, T + 2);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // Register 4 q + t of tile (i, j) holds row 32 i + r, column 32 j + 8 q + 4 h
  // + t of the wave's part.
  const int m_wave = row0 + 128 * wy;
  if constexpr (!kGlu) {
    // Parked in the wave's own 32 KiB as rows of 256 bytes, 16-byte chunk c at
    // c ^ (row % 16), then written as whole lines, 4 rows an instruction.
    uint8_t* park = lds + wave * kSlot;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v16f_t v = acc[i][j];
        asm volatile("" : "+v"(v));
        const int row = 32 * i + r;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint2*>(park + row * 256 + 16 * ((4 * j + q) ^ (r & 15)) + 8 * h) =
              make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]),
                         pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
        MXFP4_FENCE();
      }
    const int ncol = col0 + 128 * wx, cols = p.N - ncol;
    uint16_t* to = static_cast<uint16_t*>(p.C) + (int64_t)m_wave * p.N + ncol;
    if (p.N % 8 == 0) {
      const int ch = lane & 15;
#pragma unroll 1
      for (int x0 = 0; x0 < 128; x0 += 16) {
        u32x4_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = x0 + 4 * k + (lane >> 4);
          v[k] = *reinterpret_cast<const u32x4_t*>(park + row * 256 + 16 * (ch ^ (row & 15)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = x0 + 4 * k + (lane >> 4);
          if (m_wave + row < p.M && 8 * ch < cols)
            __builtin_nontemporal_store(
                v[k], reinterpret_cast<u32x4_t*>(to + (int64_t)row * p.N + 8 * ch));
        }
      }
    } else {
      for (int row = 0; row < min(128, p.M - m_wave); ++row)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int col = 64 * half + lane;
          const uint16_t v = *reinterpret_cast<const uint16_t*>(
              park + row * 256 + 16 * ((col >> 3) ^ (row & 15)) + 2 * (col & 7));
          if (col < cols) to[(int64_t)row * p.N + col] = v;
        }
    }
  } else {
    // act goes to the first 64 KiB, 256 rows of 128 columns (256 bytes, chunk c
    // at c ^ (row % 16)); g and then u, where they are wanted, pass through the
    // wave's own 16 KiB behind it (128 bytes a row, chunk c at c ^ (row % 8)).
    const int ncol = col0 + 64 * wx;
    uint8_t* own = lds + 2 * kSlot + wave * 16384;
    if (p.gu) {
#pragma unroll
      for (int up = 0; up < 2; ++up) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v16f_t v = acc[i][2 * e + up];
            asm volatile("" : "+v"(v));
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint2*>(own + (32 * i + r) * 128 + 16 * ((4 * e + q) ^ (r & 7)) +
                                        8 * h) =
                  make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]),
                             pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
            MXFP4_FENCE();
          }
        uint16_t* to = p.gu + (int64_t)m_wave * 2 * p.N + up * (int64_t)p.N + ncol;
        const int ch = lane & 7;
#pragma unroll 1
        for (int x0 = 0; x0 < 128; x0 += 32) {
          u32x4_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = x0 + 8 * k + (lane >> 3);
            v[k] = *reinterpret_cast<const u32x4_t*>(own + row * 128 + 16 * (ch ^ (row & 7)));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = x0 + 8 * k + (lane >> 3);
            if (m_wave + row < p.M)
              __builtin_nontemporal_store(
                  v[k], reinterpret_cast<u32x4_t*>(to + (int64_t)row * 2 * p.N + 8 * ch));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        v16f_t g = acc[i][2 * e], u = acc[i][2 * e + 1];
        asm volatile("" : "+v"(g), "+v"(u));
        const int row = 32 * i + r;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] = silu_f32(g[4 * q + t]) * u[4 * q + t];
          *reinterpret_cast<uint2*>(lds + (128 * wy + row) * 256 +
                                    16 * ((8 * wx + 4 * e + q) ^ (r & 15)) + 8 * h) =
              make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
        MXFP4_FENCE();
      }
    __syncthreads();
    // The quantize of a row's 128 activations: 16 lanes, as quantize_fp8.hip.
    const int ch = lane & 15;
    uint16_t* act_bf16 = static_cast<uint16_t*>(p.C);
#pragma unroll 1
    for (int x0 = 0; x0 < 64; x0 += 16) {
      u32x4_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 64 * wave + x0 + 4 * k + (lane >> 4);
        v[k] = *reinterpret_cast<const u32x4_t*>(lds + row * 256 + 16 * (ch ^ (row & 15)));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int m = row0 + 64 * wave + x0 + 4 * k + (lane >> 4);
        const uint32_t byte = fp8_row_scale<kE4M3>(v[k]);
        const uint2 code = fp8_encode_chunk<kE4M3>(v[k], fp8_scale_value(byte));
        if (m < p.M) {
          *reinterpret_cast<uint2*>(act.codes + (int64_t)m * p.N + col0 + 8 * ch) = code;
          if (ch == 0) act.scales[(int64_t)m * (p.N / kFp8Block) + tn] = (uint8_t)byte;
          if (act_bf16)
            __builtin_nontemporal_store(
                v[k], reinterpret_cast<u32x4_t*>(act_bf16 + (int64_t)m * p.N + col0 + 8 * ch));
        }
      }
    }
  }
}

template <Fp8Out kOut, Fp8Type kA, bool kRowsB>
hipError_t launch(const Fp8GemmArgs& a, const Fp8ActOut& act, hipStream_t stream) {
  constexpr int kCols = kOut == kFp8Glu ? kTile / 2 : kTile;
  const int64_t tiles_m = ((int64_t)a.M + kTile - 1) / kTile;
  const int64_t tiles_n = ((int64_t)a.N + kCols - 1) / kCols;
  const dim3 grid = grid_of(tiles_m * tiles_n, kThreads);
  if (a.K % kFp8Block != 0)
    hipLaunchKernelGGL((gemm_fp8_tile_kernel<kOut, kA, kRowsB, true>), grid, dim3(kThreads), 0,
                       stream, a, (int)tiles_m, (int)tiles_n, act);
  else
    hipLaunchKernelGGL((gemm_fp8_tile_kernel<kOut, kA, kRowsB, false>), grid, dim3(kThreads), 0,
                       stream, a, (int)tiles_m, (int)tiles_n, act);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp8_tile(const Fp8GemmArgs& a, Fp8Out out, Fp8Type a_type,
                                const Fp8ActOut& act, hipStream_t stream) {
  if (out == kFp8Glu) return launch<kFp8Glu, kE4M3, false>(a, act, stream);
  if (a_type == kE4M3)
    return a.b_shift ? launch<kFp8Bf16, kE4M3, false>(a, act, stream)
                     : launch<kFp8Bf16, kE4M3, true>(a, act, stream);
  return a.b_shift ? launch<kFp8Bf16, kE5M2, false>(a, act, stream)
                   : launch<kFp8Bf16, kE5M2, true>(a, act, stream);
}

}  // namespace mxfp4
