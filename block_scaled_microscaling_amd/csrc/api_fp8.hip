// C ABI of the FP8 operators (declared in include/mxfp4_fp8.h).
//
// As in api.hip, every entry point validates all of its arguments before
// enqueuing anything, needs a gfx950 device to be current and maps HIP
// launch errors to MXFP4_ELAUNCH.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxfp4_fp8.h"
#include "fp8.h"

namespace {

using mxfp4::Fp8Type;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 256;  // a tile past the end stays in 32 bits
constexpr int64_t kMaxK = int64_t(1) << 24;
constexpr int64_t kMaxBytes = int64_t(1) << 40;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a * b * c < kMaxBytes for non-negative factors, without overflowing.
bool below_max_bytes(int64_t a, int64_t b, int64_t c = 1) {
  int64_t ab = 0, abc = 0;
  if (__builtin_mul_overflow(a, b, &ab) || __builtin_mul_overflow(ab, c, &abc)) return false;
  return abc < kMaxBytes;
}

bool valid_rows(int64_t n) { return n >= 1 && n <= kMaxDim; }
bool valid_k(int64_t k) { return k >= 16 && k % 16 == 0 && k <= kMaxK; }
bool valid_type(int t) { return t == MXFP4_FP8_E4M3 || t == MXFP4_FP8_E5M2; }
bool valid_scale(int t) { return t == MXFP4_SCALE_UE8M0 || t == MXFP4_SCALE_FP32; }
bool aligned_scales(const void* p, int t) { return t == MXFP4_SCALE_UE8M0 || aligned(p, 4); }
Fp8Type fp8_type(int t) { return t == MXFP4_FP8_E4M3 ? mxfp4::kE4M3 : mxfp4::kE5M2; }
int64_t blocks(int64_t n) { return (n + mxfp4::kFp8Block - 1) / mxfp4::kFp8Block; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

int launch_status(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ELAUNCH; }

int quantize(const void* x, int64_t ldx, int64_t M, int64_t K, int64_t block_rows, int code_type,
             int scale_type, void* codes, void* scales, bool both, void* codes_t, void* scales_t,
             void* stream) {
  if (!x || !codes || !scales || (both && (!codes_t || !scales_t))) return MXFP4_EINVAL;
  if (!valid_rows(M) || !valid_k(K) || (both && M > kMaxK)) return MXFP4_EINVAL;
  if (block_rows != 1 && block_rows != mxfp4::kFp8Block) return MXFP4_EINVAL;
  if (!valid_type(code_type) || !valid_scale(scale_type)) return MXFP4_EINVAL;
  if (M > 1 && (ldx < K || ldx % 8 != 0)) return MXFP4_EINVAL;
  if (!below_max_bytes(M, M > 1 ? ldx : K, 2) || !below_max_bytes(M, K) ||
      !below_max_bytes(up16(M), K) || !below_max_bytes(M, blocks(K), 4))
    return MXFP4_EINVAL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(codes_t, 16) ||
      !aligned_scales(scales, scale_type) || !aligned_scales(scales_t, scale_type))
    return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  mxfp4::Fp8QuantArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.M = (int)M;
  a.K = (int)K;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.codes_t = both ? static_cast<uint8_t*>(codes_t) : nullptr;
  a.scales_t = scales_t;
  a.scale_f32 = scale_type == MXFP4_SCALE_FP32;
  return launch_status(mxfp4::launch_quantize_fp8(a, (int)block_rows, fp8_type(code_type),
                                                  static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int mxfp4_quantize_fp8(const void* x_bf16, int64_t ldx, int64_t M, int64_t K, int64_t block_rows,
                       int code_type, int scale_type, void* codes, void* scales, void* stream) {
  return quantize(x_bf16, ldx, M, K, block_rows, code_type, scale_type, codes, scales, false,
                  nullptr, nullptr, stream);
}

int mxfp4_quantize_fp8_2d(const void* x_bf16, int64_t ldx, int64_t M, int64_t K,
                          int64_t block_rows, int code_type, int scale_type, void* codes,
                          void* scales, void* codes_t, void* scales_t, void* stream) {
  return quantize(x_bf16, ldx, M, K, block_rows, code_type, scale_type, codes, scales, true,
                  codes_t, scales_t, stream);
}

int mxfp4_gemm_fp8(const void* A_codes, int A_type, const void* A_scales, const void* B_codes,
                   const void* B_scales, int scale_type, int64_t B_block_rows, int64_t M,
                   int64_t N, int64_t K, int out_dtype, void* C, void* stream) {
  if (!A_codes || !A_scales || !B_codes || !B_scales || !C) return MXFP4_EINVAL;
  if (!valid_rows(M) || !valid_rows(N) || !valid_k(K)) return MXFP4_EINVAL;
  if (!valid_type(A_type) || !valid_scale(scale_type)) return MXFP4_EINVAL;
  if (B_block_rows != mxfp4::kFp8Block &&
      (B_block_rows != 1 || scale_type != MXFP4_SCALE_UE8M0))
    return MXFP4_EINVAL;
  if (out_dtype != MXFP4_OUT_BF16 && out_dtype != MXFP4_OUT_FP32) return MXFP4_EINVAL;
  if (!below_max_bytes(M, K) || !below_max_bytes(N, K) ||
      !below_max_bytes(M, N, out_dtype == MXFP4_OUT_FP32 ? 4 : 2))
    return MXFP4_EINVAL;
  if (!aligned(A_codes, 16) || !aligned(B_codes, 16) || !aligned(C, 16) ||
      !aligned_scales(A_scales, scale_type) || !aligned_scales(B_scales, scale_type))
    return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  mxfp4::Fp8GemmArgs a{};
  a.A = static_cast<const uint8_t*>(A_codes);
  a.As = A_scales;
  a.B = static_cast<const uint8_t*>(B_codes);
  a.Bs = B_scales;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.kblocks = (int)blocks(K);
  a.b_shift = B_block_rows == 1 ? 0 : 7;
  a.C = C;
  return launch_status(mxfp4::launch_gemm_fp8(
      a, out_dtype == MXFP4_OUT_FP32 ? mxfp4::kFp8F32 : mxfp4::kFp8Bf16, fp8_type(A_type),
      scale_type == MXFP4_SCALE_FP32, static_cast<hipStream_t>(stream)));
}

int mxfp4_gemm_fp8_swiglu_workspace(int64_t M, int64_t I, int64_t K, int64_t* bytes) {
  if (!bytes || !valid_rows(M) || !valid_k(I) || I % mxfp4::kFp8Block != 0 || !valid_k(K))
    return MXFP4_EINVAL;
  if (!below_max_bytes(M, I, 4) || !below_max_bytes(2 * I, K) || !below_max_bytes(M, K))
    return MXFP4_EINVAL;
  *bytes = mxfp4::gemm_fp8_swiglu_small(M, I, K) ? 2 * M * I : 0;
  return MXFP4_OK;
}

int mxfp4_gemm_fp8_swiglu(const void* A_codes, const void* A_scales, const void* W13_codes,
                          const void* W13_scales, int64_t M, int64_t I, int64_t K, void* codes,
                          void* scales, void* act_bf16, void* gu_bf16, void* workspace,
                          void* stream) {
  if (!A_codes || !A_scales || !W13_codes || !W13_scales || !codes || !scales) return MXFP4_EINVAL;
  int64_t bytes = 0;
  if (mxfp4_gemm_fp8_swiglu_workspace(M, I, K, &bytes) != MXFP4_OK) return MXFP4_EINVAL;
  if (bytes > 0 && !workspace) return MXFP4_EINVAL;
  if (!aligned(A_codes, 16) || !aligned(W13_codes, 16) || !aligned(codes, 16) ||
      !aligned(act_bf16, 16) || !aligned(gu_bf16, 16) || !aligned(workspace, 16))
    return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  mxfp4::Fp8GemmArgs a{};
  a.A = static_cast<const uint8_t*>(A_codes);
  a.As = A_scales;
  a.B = static_cast<const uint8_t*>(W13_codes);
  a.Bs = W13_scales;
  a.M = (int)M;
  a.N = (int)I;
  a.K = (int)K;
  a.kblocks = (int)blocks(K);
  a.b_shift = 7;
  a.C = act_bf16;
  a.gu = static_cast<uint16_t*>(gu_bf16);
  return launch_status(mxfp4::launch_gemm_fp8_swiglu(
      a, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), workspace,
      static_cast<hipStream_t>(stream)));
}

int mxfp4_swiglu_fp8_backward(const void* dact_bf16, const void* gu_bf16, int64_t M, int64_t I,
                              int code_type, void* codes, void* scales, void* codes_t,
                              void* scales_t, void* stream) {
  if (!dact_bf16 || !gu_bf16 || !codes || !scales || !codes_t || !scales_t) return MXFP4_EINVAL;
  if (M < 1 || M > kMaxK || !valid_k(I) || I % mxfp4::kFp8Block != 0) return MXFP4_EINVAL;
  if (!valid_type(code_type) || !below_max_bytes(up16(M), I, 4)) return MXFP4_EINVAL;
  if (!aligned(dact_bf16, 16) || !aligned(gu_bf16, 16) || !aligned(codes, 16) ||
      !aligned(codes_t, 16))
    return MXFP4_EALIGN;
  if (!mxfp4_available()) return MXFP4_EUNSUPPORTED;
  mxfp4::SwigluBackwardArgs a{};
  a.dact = static_cast<const uint16_t*>(dact_bf16);
  a.gu = static_cast<const uint16_t*>(gu_bf16);
  a.M = (int)M;
  a.I = (int)I;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.codes_t = static_cast<uint8_t*>(codes_t);
  a.scales_t = static_cast<uint8_t*>(scales_t);
  return launch_status(mxfp4::launch_swiglu_fp8_backward(a, fp8_type(code_type),
                                                         static_cast<hipStream_t>(stream)));
}

}  // extern "C"
