// y = x dq(W)^T for a few BF16 rows x and an MXFP4 weight W [N, K].
//
// Mathematics: y[m, n] = sum_k x[m, k] E2M1(code[n, k]) 2^(scale[n, k/32] -
// 127). A weight value has two significand bits, so it is exact in BF16 and
// every product is exact in FP32; only the FP32 sums round.
//
// What bounds it: the weight's 17/32 byte per element, read once, for 2 M flop
// per element: HBM; from about 8 rows on also the re-reads of x from L2, once
// a workgroup. 1 x 8192 x 8192 8.0 us (4.5 TB/s), 8 x 4096 x 14336 9.2 us, 16
// x 28672 x 4096 15.5 us, 1 x 28672 x 4096 11.0 us (5.7 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fewtoken.h"

namespace mxfp4 {
namespace {

// Workgroups along N: a grid's extent counts threads in 32 bits, so rows of
// kGridX workgroups are stacked along z.
constexpr int64_t kGridX = 1 << 20;

__device__ __forceinline__ int64_t block_n() {
  return (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
}

dim3 grid_n(int64_t blocks, int y) {
  return blocks <= kGridX ? dim3((uint32_t)blocks, y)
                          : dim3((uint32_t)kGridX, y, (uint32_t)((blocks + kGridX - 1) / kGridX));
}

// One row of x. A wave takes 64 blocks (2048 k) of four weight rows, a block
// a lane: each load is 1 KiB of one row, all of them are issued at once, and
// the waves of a workgroup are the segments of K. Four rows rather than 8 or
// 16: 8192 x 8192 7.4 us against 7.7 and 8.4; the MFMA kernel below 9.4.
constexpr int kOneRows = 4;

template <bool kOutFp32>
__global__ __launch_bounds__(64 * kMaxWaves) void gemv_one_kernel(
    const uint8_t* __restrict__ x, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int N, int KB, void* __restrict__ y) {
  __shared__ float red[kMaxWaves * kOneRows];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int64_t n0 = block_n() * kOneRows;
  if (n0 >= N) return;
  float acc[kOneRows] = {};
  for (int s = wave; s * 64 < KB; s += waves) {
    const bool in = s * 64 + lane < KB;
    const int b = in ? s * 64 + lane : KB - 1;
    u32x4_t w[kOneRows], xv[4];
    uint32_t byte[kOneRows];
#pragma unroll
    for (int r = 0; r < kOneRows; ++r) {
      const int64_t n = min(n0 + r, (int64_t)N - 1);  // rows past the end are not stored
      w[r] = *reinterpret_cast<const u32x4_t*>(codes + n * KB * 16 + (int64_t)b * 16);
      byte[r] = scales[n * KB + b];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      xv[q] = *reinterpret_cast<const u32x4_t*>(x + (int64_t)b * 64 + 16 * q);
    if (!in) {
#pragma unroll
      for (int q = 0; q < 4; ++q) xv[q] = u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int r = 0; r < kOneRows; ++r)
      acc[r] = dot_block(w[r], scale_of_byte(in ? byte[r] : 127u), xv, acc[r]);
  }
  const float sum = sum_four_rows(acc);
  if ((lane & 15) == 0) red[wave * kOneRows + (lane >> 4)] = sum;
  __syncthreads();
  if (threadIdx.x < kOneRows && n0 + threadIdx.x < N) {
    float v = red[threadIdx.x];
    for (int w = 1; w < waves; ++w) v += red[w * kOneRows + threadIdx.x];
    store_y<kOutFp32>(y, n0 + threadIdx.x, v);
  }
}

// The same for K <= 32 kLanes: 256 / kLanes weight rows a wave (11968 x 448
// 3.3 -> 2.3 us, 11328 x 928 3.3 -> 2.7, 19321 x 1728 5.2 -> 4.5).
template <int kLanes, bool kOutFp32>
__global__ __launch_bounds__(64 * kShortWaves) void gemv_one_short_kernel(
    const uint8_t* __restrict__ x, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int N, int KB, void* __restrict__ y) {
  constexpr int kGroups = 64 / kLanes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t n0 = (block_n() * kShortWaves + wave) * 4 * kGroups;
  if (n0 >= N) return;
  codes += n0 * KB * 16;
  scales += n0 * KB;
  const int last = (int)min((int64_t)N - 1 - n0, (int64_t)(4 * kGroups - 1));
  const int j = lane / kLanes;
  const bool in = lane % kLanes < KB;
  const uint32_t b = in ? lane % kLanes : KB - 1;
  u32x4_t w[4], xv[4];
  uint32_t byte[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t row = min(r * kGroups + j, last);  // rows past the end are not stored
    w[r] = *reinterpret_cast<const u32x4_t*>(codes + (row * KB + b) * 16);
    byte[r] = scales[row * KB + b];
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    xv[q] = *reinterpret_cast<const u32x4_t*>(x + b * 64 + 16 * q);
  if (!in) {
#pragma unroll
    for (int q = 0; q < 4; ++q) xv[q] = u32x4_t{0u, 0u, 0u, 0u};
  }
  float v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    v[r] = dot_block(w[r], scale_of_byte(in ? byte[r] : 127u), xv, 0.0f);
  if constexpr (kLanes == 64) {
    const float sum = sum_four_rows(v);
    if ((lane & 15) == 0 && (lane >> 4) <= last) store_y<kOutFp32>(y, n0 + (lane >> 4), sum);
  } else if constexpr (kLanes == 32) {
    // Even 16 lanes: rows 0 and 2 of the lane's, odd ones: rows 1 and 3.
    v[0] = sum16(merge16(v[0], v[1]));
    v[1] = sum16(merge16(v[2], v[3]));
    const int r = 2 * (lane & 1) + ((lane >> 4) & 1), n = r * kGroups + j;
    if ((lane & 15) < 2 && n <= last) store_y<kOutFp32>(y, n0 + n, lane & 1 ? v[1] : v[0]);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = sum16(v[r]);
    const int r = lane & 3, n = r * kGroups + j;
    const float lo = r & 1 ? v[1] : v[0], hi = r & 1 ? v[3] : v[2];
    if ((lane & 15) < 4 && n <= last) store_y<kOutFp32>(y, n0 + n, r & 2 ? hi : lo);
  }
}

// Several rows of x: a workgroup owns T tiles of 16 weight rows and up to 16
// rows of x, its waves take the units of 256 k in turn, and the partial tiles
// are summed in LDS in wave order.
template <int T, int XL, bool kAhead, bool kOutFp32>
__global__ __launch_bounds__(64 * kMaxWaves) void gemv_few_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int M, int N, int KB, void* __restrict__ y) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int64_t n0 = block_n() * (T * kFewTile);
  if (n0 >= N) return;
  const int m0 = blockIdx.y * kFewTile;
  const int last = (int)min((int64_t)N - 1 - n0, (int64_t)(T * kFewTile - 1));
  const uint8_t* wc[T];
  const uint8_t* ws[T];
  v4f_t acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    wc[t] = codes + n0 * KB * 16;
    ws[t] = scales + n0 * KB;
    acc[t] = v4f_t{};
  }
  BfRows<XL> rows;
#pragma unroll
  for (int i = 0; i < XL; ++i)
    rows.p[i] = x + (int64_t)min(m0 + 4 * i + (lane >> 4), M - 1) * ldx * 2 + (lane & 3) * 16;
  // Rows past the end re-read the last one; they are not stored.
  few_stream<T, kAhead>(wc, ws, [&](int t, int r) { return min(kFewTile * t + r, last); }, rows, KB,
                        wave, waves, lds + wave * few_lds_bytes<T, BfRows<XL>>(), acc);
  __syncthreads();
  auto* red = reinterpret_cast<float*>(lds);
  // Output (row 4 g + v, column c) at 64 v + 16 g + c of the wave's part.
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) red[(t * waves + wave) * 256 + v * 64 + lane] = acc[t][v];
  __syncthreads();
  for (int i = threadIdx.x; i < T * 256; i += blockDim.x) {
    // Row i % 16 of column i / 16 % 16, so a token's rows store together.
    const int t = i >> 8, r = i & 15, c = (i >> 4) & 15;
    const float* part = red + t * waves * 256 + (r & 3) * 64 + (r >> 2) * 16 + c;
    float v = part[0];
    for (int w = 1; w < waves; ++w) v += part[w * 256];
    if (kFewTile * t + r <= last && c < 4 * XL && m0 + c < M)
      store_y<kOutFp32>(y, (int64_t)(m0 + c) * N + n0 + kFewTile * t + r, v);
  }
}

template <int T, int XL, bool kAhead>
hipError_t launch_few(const uint8_t* x, int64_t ldx, const uint8_t* codes, const uint8_t* scales,
                      int M, int N, int KB, bool out_fp32, void* y, hipStream_t stream) {
  const int waves = even_waves((KB + kUnitBlocks - 1) / kUnitBlocks, kMaxWaves);
  // The partial tiles (T KiB a wave) take the place of what was streamed.
  static_assert(few_lds_bytes<T, BfRows<XL>>() >= T * 1024, "");
  const int lds = waves * few_lds_bytes<T, BfRows<XL>>();
  const dim3 grid = grid_n(((int64_t)N + T * kFewTile - 1) / (T * kFewTile),
                           (M + kFewTile - 1) / kFewTile);
  const auto kernel = out_fp32 ? gemv_few_kernel<T, XL, kAhead, true>
                               : gemv_few_kernel<T, XL, kAhead, false>;
  // The limit is the process's, not the call's: every call sets the same one,
  // so that none can lower it between another thread's set and launch.
  constexpr int kMostLds = kMaxWaves * few_lds_bytes<T, BfRows<XL>>();
  if (kMostLds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kMostLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), lds, stream, x, ldx, codes, scales, M, N, KB,
                     y);
  return hipGetLastError();
}

// Several rows of x and many weight rows: the workgroup's waves are four tiles
// of 16 weight rows times two parts of K, and the four waves of a part share
// each unit of x, of which each loads a quarter, in LDS. So x is read from L2
// once for 64 weight rows and a wave's registers hold one tile's weights and
// little of x, which leaves room for three workgroups a CU. x is double-
// buffered: one barrier a unit. 16 rows x 28672 x 4096: one part of K
// 15.6 us, two 14.8, four 18.9; two tiles and four parts 23.5, eight tiles
// 15.2, four tiles with two units in flight 16.2.
constexpr int kShareParts = 2;

template <int XL, bool kOutFp32>
__global__ __launch_bounds__(64 * kShareTiles * kShareParts) void gemv_share_kernel(
    const uint8_t* __restrict__ x, int64_t ldx, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int M, int N, int KB, void* __restrict__ y) {
  constexpr int kColumns = 4 * XL;
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int parts = (blockDim.x >> 6) / kShareTiles;
  const int tile = wave % kShareTiles;
  const int64_t n0 = block_n() * (kShareTiles * kFewTile);
  if (n0 >= N) return;
  const int m0 = blockIdx.y * kFewTile;
  // Rows past the end re-read the last one; they are not stored.
  const int last = (int)min((int64_t)N - 1 - n0, (int64_t)(kShareTiles * kFewTile - 1));
  v4f_t acc[1] = {v4f_t{}};
  share_stream<XL, 64>(
      codes + n0 * KB * 16, scales + n0 * KB,
      [&](int r) { return min(kFewTile * tile + r, last); },
      [&](int r) { return x + (int64_t)min(m0 + r, M - 1) * ldx * 2 + (lane & 3) * 16; }, KB, tile,
      wave / kShareTiles, parts, lds, acc);
  __syncthreads();
  auto* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave * 256 + v * 64 + lane] = acc[0][v];
  __syncthreads();
  for (int i = threadIdx.x; i < kShareTiles * 256; i += blockDim.x) {
    // Row i % 16 of column i / 16 % 16, so a token's rows store together.
    const int t = i >> 8, r = i & 15, c = (i >> 4) & 15;
    const float* p = red + t * 256 + (r & 3) * 64 + (r >> 2) * 16 + c;
    float v = p[0];
    for (int q = 1; q < parts; ++q) v += p[q * kShareTiles * 256];
    if (kFewTile * t + r <= last && c < kColumns && m0 + c < M)
      store_y<kOutFp32>(y, (int64_t)(m0 + c) * N + n0 + kFewTile * t + r, v);
  }
}

template <int XL>
hipError_t launch_share(const uint8_t* x, int64_t ldx, const uint8_t* codes, const uint8_t* scales,
                        int M, int N, int KB, bool out_fp32, void* y, hipStream_t stream) {
  const int parts = KB > kUnitBlocks ? kShareParts : 1;
  const int streamed = share_lds_bytes<XL>(parts);
  const int lds = streamed > parts * kShareTiles * 1024 ? streamed : parts * kShareTiles * 1024;
  static_assert(share_lds_bytes<4>(kShareParts) <= 65536, "");
  const int64_t rows = kShareTiles * kFewTile;
  const dim3 grid = grid_n(((int64_t)N + rows - 1) / rows, (M + kFewTile - 1) / kFewTile);
  const auto kernel = out_fp32 ? gemv_share_kernel<XL, true> : gemv_share_kernel<XL, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(64 * kShareTiles * parts), lds, stream, x, ldx, codes,
                     scales, M, N, KB, y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv(const void* x, int64_t ldx, const void* codes, const void* scales, int M,
                       int N, int K, bool out_fp32, void* y, hipStream_t stream) {
  const auto* xb = static_cast<const uint8_t*>(x);
  const auto* wc = static_cast<const uint8_t*>(codes);
  const auto* ws = static_cast<const uint8_t*>(scales);
  const int KB = K / 32;
  if (M == 1 && KB <= 64) {
    const int rows = (KB <= 16 ? 16 : KB <= 32 ? 8 : 4) * kShortWaves;
    const auto short_kernel = [&](auto lanes) {
      constexpr int kLanes = decltype(lanes)::value;
      return out_fp32 ? gemv_one_short_kernel<kLanes, true> : gemv_one_short_kernel<kLanes, false>;
    };
    hipLaunchKernelGGL(KB <= 16   ? short_kernel(std::integral_constant<int, 16>{})
                       : KB <= 32 ? short_kernel(std::integral_constant<int, 32>{})
                                  : short_kernel(std::integral_constant<int, 64>{}),
                       grid_n(((int64_t)N + rows - 1) / rows, 1), dim3(64 * kShortWaves), 0, stream,
                       xb, wc, ws, N, KB, y);
    return hipGetLastError();
  }
  if (M == 1) {
    const dim3 grid = grid_n(((int64_t)N + kOneRows - 1) / kOneRows, 1);
    const dim3 threads(64 * even_waves((KB + 63) / 64, kMaxWaves));
    if (out_fp32)
      hipLaunchKernelGGL((gemv_one_kernel<true>), grid, threads, 0, stream, xb, wc, ws, N, KB, y);
    else
      hipLaunchKernelGGL((gemv_one_kernel<false>), grid, threads, 0, stream, xb, wc, ws, N, KB, y);
    return hipGetLastError();
  }
  // With 64 weight rows a workgroup in at least 160 of them (5/8 of the CUs)
  // the waves share x: 16 rows x 28672 x 4096 15.2 against 17.9 us, 8 rows
  // 13.5 against 15.8, 16 x 16384 x 288 3.7 against 4.4, 64 x 14336 x 4096
  // 24.4 against 27.3, 8 x 10240 x 4096 (160 workgroups) 8.8 against 9.3; with
  // fewer they are too few (16 x 8192 x 8192, 128, 15.3 against 11.1). A little
  // over one workgroup a CU is the rule's worst (8 x 20000 x 1024, 313, 5.4
  // against 5.0). Up to four rows there is little x to share: 4 x 65536 x 4096
  // 30.0 against 33.4, but 4 x 40000 x 4096 19.3 against 17.9, 4 x 12288 x
  // 4096 8.8 against 7.7 and 3 x 20000 x 256 3.6 against 3.0.
  const int64_t groups = (M + kFewTile - 1) / kFewTile;
  const int64_t blocks = ((int64_t)N + kShareTiles * kFewTile - 1) / (kShareTiles * kFewTile);
  if (M > 4 && KB >= kUnitBlocks && blocks * groups >= 160)
    return M <= 8 ? launch_share<2>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream)
                  : launch_share<4>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream);
  // Two tiles a workgroup halve the reads of x from L2 but also the
  // workgroups: from 384 tiles on (1.5 a CU) they pay (5 rows x 6177 x 7968
  // 8.8 against 9.6 us, 16 x 8192 x 8192 10.9 against 13.1), below not (8 x
  // 4096 x 14336 10.7 against 8.8, 16 x 4096 x 14336 12.5 against 10.7). Up to
  // four rows x is small and one tile is never slower by more than 1%.
  // Loading ahead pays where a wave has few others beside it and few
  // registers to spend (8 x 4096 x 14336 8.8 against 9.5 us), not with two
  // tiles or 16 rows of x (8 x 8192 x 8192 10.2 against 10.0, 16 x 6177 x 7968
  // 11.6 against 11.3).
  const int64_t tiles = ((int64_t)N + kFewTile - 1) / kFewTile * groups;
  if (M <= 4) return launch_few<1, 1, true>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream);
  if (tiles < 384)
    return M <= 8 ? launch_few<1, 2, true>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream)
                  : launch_few<1, 4, false>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream);
  return M <= 8 ? launch_few<2, 2, false>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream)
                : launch_few<2, 4, false>(xb, ldx, wc, ws, M, N, KB, out_fp32, y, stream);
}

}  // namespace mxfp4
