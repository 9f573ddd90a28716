// C ABI of the few-token operators (declared in include/mxfp4_fewtoken.h).
//
// As in api.hip, every entry point validates all of its arguments before
// enqueuing anything, needs a gfx950 device to be current and maps HIP
// launch errors to MXFP4_ELAUNCH.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxfp4_fewtoken.h"
#include "fewtoken.h"

namespace {

constexpr int64_t kMaxDim = 2147483647;
constexpr int64_t kMaxBytes = int64_t(1) << 40;
constexpr int64_t kMaxK = int64_t(1) << 24;
constexpr int64_t kMaxGemvM = 65535LL * 16;  // 16-token groups in the grid's y extent
constexpr int64_t kMaxMoeDim = int64_t(1) << 20;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 32;
constexpr int64_t kMaxRouteT = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b * c < kMaxBytes for non-negative factors, without overflowing.
bool below_max_bytes(int64_t a, int64_t b, int64_t c = 1) {
  int64_t ab = 0, abc = 0;
  if (__builtin_mul_overflow(a, b, &ab) || __builtin_mul_overflow(ab, c, &abc)) return false;
  return abc < kMaxBytes;
}

// Rows of BF16 activations: `rows` of `cols` elements, ldx elements apart.
bool valid_rows(int64_t rows, int64_t cols, int64_t ldx) {
  if (rows == 1) return true;
  return ldx >= cols && ldx % 8 == 0 && below_max_bytes(rows, ldx, 2);
}

bool valid_out(int out_dtype) {
  return out_dtype == MXFP4_OUT_BF16 || out_dtype == MXFP4_OUT_FP32;
}

int64_t out_bytes(int out_dtype) { return out_dtype == MXFP4_OUT_FP32 ? 4 : 2; }

int launch_status(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ELAUNCH; }

}  // namespace

extern "C" {

int mxfp4_gemv(const void* x_bf16, int64_t ldx, const void* W_codes, const void* W_scales,
               int64_t M, int64_t N, int64_t K, int out_dtype, void* y, void* stream) {
  if (!x_bf16 || !W_codes || !W_scales || !y) return MXFP4_EINVAL;
  if (M < 1 || M > kMaxGemvM || N < 1 || N > kMaxDim || K < 32 || K % 32 != 0 || K > kMaxK)
    return MXFP4_EINVAL;
  if (!valid_out(out_dtype) || !valid_rows(M, K, ldx)) return MXFP4_EINVAL;
  if (!below_max_bytes(N, K / 2) || !below_max_bytes(M, N, out_bytes(out_dtype)))
    return MXFP4_EINVAL;
  if (!aligned(x_bf16, 16) || !aligned(W_codes, 16) || !aligned(y, 4)) return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  return launch_status(mxfp4::launch_gemv(x_bf16, ldx, W_codes, W_scales, (int)M, (int)N, (int)K,
                                          out_dtype == MXFP4_OUT_FP32, y,
                                          static_cast<hipStream_t>(stream)));
}

int mxfp4_moe_route_workspace(int64_t T, int64_t H, int64_t E, int64_t* bytes) {
  if (!bytes || T < 1 || T > kMaxRouteT || E < 1 || E > kMaxExperts) return MXFP4_EINVAL;
  if (H < 8 || H % 8 != 0 || H > kMaxK) return MXFP4_EINVAL;
  *bytes = mxfp4::moe_route_workspace_bytes(T, H, E);
  return MXFP4_OK;
}

int mxfp4_moe_route(const void* x_bf16, int64_t ldx, const void* router_bf16, int64_t T, int64_t H,
                    int64_t E, int64_t top_k, int renormalize, void* ids, void* weights,
                    void* workspace, void* stream) {
  if (!x_bf16 || !router_bf16 || !ids || !weights) return MXFP4_EINVAL;
  int64_t bytes = 0;
  if (mxfp4_moe_route_workspace(T, H, E, &bytes) != MXFP4_OK) return MXFP4_EINVAL;
  if (bytes > 0 && !workspace) return MXFP4_EINVAL;
  if (top_k < 1 || top_k > kMaxTopK || top_k > E) return MXFP4_EINVAL;
  if (renormalize != 0 && renormalize != 1) return MXFP4_EINVAL;
  if (!valid_rows(T, H, ldx)) return MXFP4_EINVAL;
  if (!aligned(x_bf16, 16) || !aligned(router_bf16, 16) || !aligned(ids, 4) ||
      !aligned(weights, 4) || !aligned(workspace, 16))
    return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  return launch_status(mxfp4::launch_moe_route(
      x_bf16, ldx, router_bf16, (int)T, (int)H, (int)E, (int)top_k, renormalize == 1,
      static_cast<int32_t*>(ids), static_cast<float*>(weights), static_cast<double*>(workspace),
      static_cast<hipStream_t>(stream)));
}

int mxfp4_moe_workspace(int64_t T, int64_t H, int64_t I, int64_t top_k, int64_t* bytes) {
  if (!bytes || T < 1 || top_k < 1 || top_k > kMaxTopK || T > mxfp4::kMaxPairs ||
      T * top_k > mxfp4::kMaxPairs)
    return MXFP4_EINVAL;
  if (H < 32 || H % 32 != 0 || H > kMaxMoeDim || I < 32 || I % 32 != 0 || I > kMaxMoeDim)
    return MXFP4_EINVAL;
  // One token: the pairs' activations, FP32. Several: three BF16 pieces of the
  // activations and the pairs' parts of y, FP32.
  *bytes = T * top_k * (T > 1 ? 6 * I + 4 * H : 4 * I);
  return MXFP4_OK;
}

int mxfp4_moe(const void* x_bf16, int64_t ldx, const void* ids, const void* weights,
              const void* W13_codes, const void* W13_scales, const void* W2_codes,
              const void* W2_scales, int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k,
              int out_dtype, void* y, void* workspace, void* stream) {
  if (!x_bf16 || !ids || !weights || !W13_codes || !W13_scales || !W2_codes || !W2_scales || !y ||
      !workspace)
    return MXFP4_EINVAL;
  int64_t bytes = 0;
  if (mxfp4_moe_workspace(T, H, I, top_k, &bytes) != MXFP4_OK) return MXFP4_EINVAL;
  if (E < 1 || E > kMaxExperts) return MXFP4_EINVAL;
  if (!valid_out(out_dtype) || !valid_rows(T, H, ldx)) return MXFP4_EINVAL;
  if (!below_max_bytes(E, I, H)) return MXFP4_EINVAL;
  if (!aligned(x_bf16, 16) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(W13_codes, 16) || !aligned(W2_codes, 16) || !aligned(y, 4) ||
      !aligned(workspace, 16))
    return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  return launch_status(mxfp4::launch_moe(
      x_bf16, ldx, static_cast<const int32_t*>(ids), static_cast<const float*>(weights),
      W13_codes, W13_scales, W2_codes, W2_scales, (int)T, (int)H, (int)I, (int)E, (int)top_k,
      out_dtype == MXFP4_OUT_FP32, y, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
