// Tensor layer of the few-token and FP8 operators: checks torch tensors,
// allocates outputs and workspaces from torch's allocator and calls the C ABI
// (include/mxfp4_fewtoken.h, include/mxfp4_fp8.h) on torch's current stream or
// a given one.
//
// These calls run once per layer and token, where the host's time counts: the
// same checks written in Python over ctypes cost 11.5 us a gemv, of which the
// launch itself is 3.4. Each function returns its outputs, or the C ABI's
// status as an int when it is not 0; a wrong argument raises TypeError or
// ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/mxfp4_fewtoken.h"
#include "../../include/mxfp4_fp8.h"

namespace {

std::string dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case at::kFloat8_e5m2: return "torch.float8_e5m2";
    default: return std::string("torch ") + c10::toString(t);
  }
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void check_dtype(const at::Tensor& t, const char* name, at::ScalarType dtype) {
  TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " must be ", dtype_name(dtype), ", got ",
                   dtype_name(t.scalar_type()));
}

// A 2-D BF16 tensor on the current device whose rows are each contiguous, ld
// elements apart (a slice of a larger activation).
struct Rows {
  const at::Tensor& t;
  int64_t rows, cols, ld;
  c10::DeviceIndex device;
};

Rows rows_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  check_dtype(t, name, at::kBFloat16);
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must be 2-D");
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a device tensor");
  const c10::DeviceIndex device = t.get_device();
  TORCH_CHECK_VALUE(device == c10::hip::current_device(), name, " must be on the current device");
  const int64_t cols = t.size(1);
  TORCH_CHECK_VALUE(t.stride(1) == 1 || cols <= 1, name, "'s rows must be contiguous");
  return {t, t.size(0), cols, t.stride(0), device};
}

const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType dtype,
                          std::initializer_list<int64_t> shape, c10::DeviceIndex device) {
  const at::Tensor& t = tensor(o, name);
  check_dtype(t, name, dtype);
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a device tensor");
  const at::IntArrayRef want(shape.begin(), shape.size());
  TORCH_CHECK_VALUE(t.sizes() == want, name, " must have shape ", shape_text(want), ", got ",
                    shape_text(t.sizes()));
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous (row-major)");
  TORCH_CHECK_VALUE(t.get_device() == device, name, " must be on the current device");
  return t;
}

// Size d of a tensor that must have `dims` dimensions (checked before its
// other sizes give the shapes of the rest).
int64_t size_of(PyObject* o, const char* name, int64_t dims, int64_t d) {
  const at::Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.dim() == dims, name, " must be ", dims, "-D");
  return t.size(d);
}

struct Stream {
  void* handle;
  std::optional<c10::Stream> given;

  // Memory of the call's stream: a block of another stream's may still be
  // read or written by what that stream has queued. A given stream's output is
  // meant for the current one, which torch waits for before it hands the
  // memory out again.
  at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType dtype) const {
    if (!given) return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
    const c10::StreamGuard guard(*given);
    at::Tensor t = at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
    if (guard.original_stream() != *given) t.record_stream(guard.original_stream());
    return t;
  }
};

Stream stream_of(PyObject* o, c10::DeviceIndex device) {
  if (o == Py_None) return {c10::hip::getCurrentHIPStream(device).stream(), std::nullopt};
  TORCH_CHECK_TYPE(PyObject_IsInstance(o, reinterpret_cast<PyObject*>(THPStreamClass)) == 1,
                   "stream must be a torch.cuda.Stream");
  const auto* s = reinterpret_cast<THPStream*>(o);
  TORCH_CHECK_VALUE(s->device_index == device, "stream must be of the current device");
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw python_error();
  void* handle = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!handle && PyErr_Occurred()) throw python_error();
  return {handle, c10::Stream::unpack3(s->stream_id, static_cast<c10::DeviceIndex>(s->device_index),
                                       static_cast<c10::DeviceType>(s->device_type))};
}

struct Output {
  at::Tensor t;
  PyObject* given;  // borrowed; the caller's own tensor, or null

  PyObject* result() {
    if (given) {
      Py_INCREF(given);
      return given;
    }
    return THPVariable_Wrap(std::move(t));
  }
};

Output output(PyObject* out, const char* name, std::initializer_list<int64_t> shape,
              at::ScalarType dtype, const Rows& x, const Stream& stream) {
  if (out == Py_None)
    return {stream.empty(at::IntArrayRef(shape.begin(), shape.size()), x.t, dtype), nullptr};
  return {checked(out, name, dtype, shape, x.device), out};
}

// The type of an output from out_dtype and out (either may be None).
at::ScalarType out_type(PyObject* out_dtype, PyObject* out) {
  at::ScalarType t = at::kBFloat16;
  if (out_dtype != Py_None) {
    TORCH_CHECK_TYPE(THPDtype_Check(out_dtype), "out_dtype must be a torch.dtype");
    t = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
  } else if (out != Py_None) {
    t = tensor(out, "out").scalar_type();
  }
  TORCH_CHECK_TYPE(t == at::kBFloat16 || t == at::kFloat,
                   "out_dtype must be torch.bfloat16 or torch.float32");
  return t;
}

int out_code(at::ScalarType t) { return t == at::kFloat ? MXFP4_OUT_FP32 : MXFP4_OUT_BF16; }

// A workspace of at least `bytes`: the caller's, or memory from torch's
// allocator that belongs to the call's stream, so that it may be given back
// once the call has been enqueued.
class Workspace {
 public:
  Workspace(PyObject* o, int64_t bytes, c10::DeviceIndex device, const Stream& stream) {
    if (o == Py_None) {
      if (bytes > 0)
        own_ = c10::hip::HIPCachingAllocator::raw_alloc_with_stream(
            bytes, static_cast<hipStream_t>(stream.handle));
      return;
    }
    const at::Tensor& t = tensor(o, "workspace");
    check_dtype(t, "workspace", at::kByte);
    TORCH_CHECK_VALUE(t.is_cuda(), "workspace must be a device tensor");
    TORCH_CHECK_VALUE(t.is_contiguous(), "workspace must be contiguous (row-major)");
    TORCH_CHECK_VALUE(t.get_device() == device, "workspace must be on the current device");
    TORCH_CHECK_VALUE(t.numel() >= bytes, "workspace must hold ", bytes, " bytes, got ",
                      t.numel());
    given_ = t.data_ptr();
  }
  ~Workspace() {
    if (own_) c10::hip::HIPCachingAllocator::raw_delete(own_);
  }
  Workspace(const Workspace&) = delete;
  Workspace& operator=(const Workspace&) = delete;
  void* ptr() const { return own_ ? own_ : given_; }

 private:
  void* own_ = nullptr;
  void* given_ = nullptr;
};

void need(Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}

// gemv(x, codes, scales, out_dtype, out, stream)
PyObject* gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 6);
  const Rows x = rows_of(a[0], "x");
  const int64_t N = size_of(a[1], "codes", 2, 0), K = x.cols;
  const at::Tensor& codes = checked(a[1], "codes", at::kByte, {N, K / 2}, x.device);
  const at::Tensor& scales = checked(a[2], "scales", at::kByte, {N, K / 32}, x.device);
  const at::ScalarType type = out_type(a[3], a[4]);
  const Stream stream = stream_of(a[5], x.device);
  Output y = output(a[4], "out", {x.rows, N}, type, x, stream);
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_gemv(x.t.const_data_ptr(), x.ld, codes.const_data_ptr(), scales.const_data_ptr(),
                  x.rows, N, K, out_code(type), y.t.data_ptr(), stream.handle);
  Py_END_ALLOW_THREADS;
  return rc ? PyLong_FromLong(rc) : y.result();
  END_HANDLE_TH_ERRORS
}

// moe_route(x, router, top_k, renormalize, ids, weights, workspace, stream)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 8);
  const Rows x = rows_of(a[0], "x");
  const int64_t T = x.rows, H = x.cols, E = size_of(a[1], "router", 2, 0);
  const at::Tensor& router = checked(a[1], "router", at::kBFloat16, {E, H}, x.device);
  const int64_t k = PyLong_AsLongLong(a[2]);
  if (k == -1 && PyErr_Occurred()) throw python_error();
  const int renormalize = PyObject_IsTrue(a[3]);
  if (renormalize < 0) throw python_error();
  int64_t bytes = 0;
  int rc = mxfp4_moe_route_workspace(T, H, E, &bytes);
  if (rc == 0 && k < 1) rc = MXFP4_EINVAL;
  if (rc) return PyLong_FromLong(rc);
  const Stream stream = stream_of(a[7], x.device);
  Output ids = output(a[4], "ids", {T, k}, at::kInt, x, stream);
  Output weights = output(a[5], "weights", {T, k}, at::kFloat, x, stream);
  const Workspace ws(a[6], bytes, x.device, stream);
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_moe_route(x.t.const_data_ptr(), x.ld, router.const_data_ptr(), T, H, E, k,
                       renormalize, ids.t.data_ptr(), weights.t.data_ptr(), ws.ptr(),
                       stream.handle);
  Py_END_ALLOW_THREADS;
  if (rc) return PyLong_FromLong(rc);
  PyObject* i = ids.result();
  PyObject* w = weights.result();
  PyObject* both = PyTuple_Pack(2, i, w);
  Py_DECREF(i);
  Py_DECREF(w);
  return both;
  END_HANDLE_TH_ERRORS
}

// moe(x, ids, weights, w13_codes, w13_scales, w2_codes, w2_scales, out_dtype,
//     out, workspace, stream)
PyObject* moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 11);
  const Rows x = rows_of(a[0], "x");
  const int64_t T = x.rows, H = x.cols;
  const int64_t k = size_of(a[1], "ids", 2, 1);
  const int64_t E = size_of(a[3], "w13_codes", 3, 0), I = 2 * size_of(a[5], "w2_codes", 3, 2);
  const at::Tensor& ids = checked(a[1], "ids", at::kInt, {T, k}, x.device);
  const at::Tensor& weights = checked(a[2], "weights", at::kFloat, {T, k}, x.device);
  const at::Tensor& c13 = checked(a[3], "w13_codes", at::kByte, {E, 2 * I, H / 2}, x.device);
  const at::Tensor& s13 = checked(a[4], "w13_scales", at::kByte, {E, 2 * I, H / 32}, x.device);
  const at::Tensor& c2 = checked(a[5], "w2_codes", at::kByte, {E, H, I / 2}, x.device);
  const at::Tensor& s2 = checked(a[6], "w2_scales", at::kByte, {E, H, I / 32}, x.device);
  const at::ScalarType type = out_type(a[7], a[8]);
  int64_t bytes = 0;
  int rc = mxfp4_moe_workspace(T, H, I, k, &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Stream stream = stream_of(a[10], x.device);
  Output y = output(a[8], "out", {T, H}, type, x, stream);
  const Workspace ws(a[9], bytes, x.device, stream);
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_moe(x.t.const_data_ptr(), x.ld, ids.const_data_ptr(), weights.const_data_ptr(),
                 c13.const_data_ptr(), s13.const_data_ptr(), c2.const_data_ptr(),
                 s2.const_data_ptr(), T, H, I, E, k, out_code(type), y.t.data_ptr(),
                 ws.ptr(), stream.handle);
  Py_END_ALLOW_THREADS;
  return rc ? PyLong_FromLong(rc) : y.result();
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------- FP8
constexpr int64_t kFp8Block = 128;
int64_t blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

// A dtype argument, or `otherwise` for None.
at::ScalarType dtype_of(PyObject* o, const char* name, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  TORCH_CHECK_TYPE(THPDtype_Check(o), name, " must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

at::ScalarType fp8_dtype(PyObject* o) {
  const at::ScalarType t = dtype_of(o, "dtype", at::kFloat8_e4m3fn);
  TORCH_CHECK_TYPE(t == at::kFloat8_e4m3fn || t == at::kFloat8_e5m2,
                   "dtype must be torch.float8_e4m3fn or torch.float8_e5m2");
  return t;
}

int fp8_code(at::ScalarType t) { return t == at::kFloat8_e5m2 ? MXFP4_FP8_E5M2 : MXFP4_FP8_E4M3; }
int scale_code(at::ScalarType t) { return t == at::kFloat ? MXFP4_SCALE_FP32 : MXFP4_SCALE_UE8M0; }

// A 2-D FP8 tensor on the current device, row-major.
struct Codes {
  const at::Tensor& t;
  int64_t rows, cols;
  at::ScalarType type;
  c10::DeviceIndex device;
};

Codes codes_of(PyObject* o, const char* name, bool e5m2) {
  const at::Tensor& t = tensor(o, name);
  const at::ScalarType type = t.scalar_type();
  TORCH_CHECK_TYPE(type == at::kFloat8_e4m3fn || (e5m2 && type == at::kFloat8_e5m2), name,
                   " must be torch.float8_e4m3fn", e5m2 ? " or torch.float8_e5m2" : "", ", got ",
                   dtype_name(type));
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must be 2-D");
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a device tensor");
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous (row-major)");
  TORCH_CHECK_VALUE(t.get_device() == c10::hip::current_device(), name,
                    " must be on the current device");
  return {t, t.size(0), t.size(1), type, t.get_device()};
}

Output output(PyObject* out, const char* name, std::initializer_list<int64_t> shape,
              at::ScalarType dtype, const Codes& x, const Stream& stream) {
  if (out == Py_None)
    return {stream.empty(at::IntArrayRef(shape.begin(), shape.size()), x.t, dtype), nullptr};
  return {checked(out, name, dtype, shape, x.device), out};
}

PyObject* tuple_of(std::initializer_list<Output*> parts) {
  PyObject* all = PyTuple_New((Py_ssize_t)parts.size());
  if (!all) throw python_error();
  Py_ssize_t i = 0;
  for (Output* p : parts) PyTuple_SET_ITEM(all, i++, p->result());
  return all;
}

bool truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw python_error();
  return t == 1;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// What both quantizers check of x and their options, and the sizes.
struct Quantize {
  Rows x;
  int64_t block;
  at::ScalarType type, scale;

  Quantize(PyObject* ox, PyObject* oblock, PyObject* odtype, PyObject* oscale)
      : x(rows_of(ox, "x")), block(integer(oblock)), type(fp8_dtype(odtype)),
        scale(dtype_of(oscale, "scale_dtype", at::kByte)) {
    TORCH_CHECK_TYPE(scale == at::kByte || scale == at::kFloat,
                     "scale_dtype must be torch.uint8 or torch.float32");
    TORCH_CHECK_VALUE(block == 1 || block == kFp8Block, "block_rows must be 1 or 128");
    TORCH_CHECK_VALUE(x.rows > 0 && x.cols > 0 && x.cols % 16 == 0,
                      "x must be [M, K] with M > 0 and K a multiple of 16, got ",
                      shape_text(x.t.sizes()));
  }
  int64_t scale_rows(int64_t rows) const { return block == 1 ? rows : blocks(rows); }
};

// quantize_fp8(x, block_rows, dtype, scale_dtype, codes, scales, stream)
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 7);
  const Quantize q(a[0], a[1], a[2], a[3]);
  const int64_t M = q.x.rows, K = q.x.cols;
  const Stream stream = stream_of(a[6], q.x.device);
  Output codes = output(a[4], "codes", {M, K}, q.type, q.x, stream);
  Output scales = output(a[5], "scales", {q.scale_rows(M), blocks(K)}, q.scale, q.x, stream);
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_quantize_fp8(q.x.t.const_data_ptr(), q.x.ld, M, K, q.block, fp8_code(q.type),
                          scale_code(q.scale), codes.t.data_ptr(), scales.t.data_ptr(),
                          stream.handle);
  Py_END_ALLOW_THREADS;
  return rc ? PyLong_FromLong(rc) : tuple_of({&codes, &scales});
  END_HANDLE_TH_ERRORS
}

// quantize_fp8_2d(x, block_rows, dtype, scale_dtype, stream)
PyObject* quantize_fp8_2d(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 5);
  const Quantize q(a[0], a[1], a[2], a[3]);
  const int64_t M = q.x.rows, K = q.x.cols;
  const Stream stream = stream_of(a[4], q.x.device);
  Output codes = output(Py_None, "codes", {M, K}, q.type, q.x, stream);
  Output scales = output(Py_None, "scales", {q.scale_rows(M), blocks(K)}, q.scale, q.x, stream);
  Output codes_t = output(Py_None, "codes_t", {K, up16(M)}, q.type, q.x, stream);
  Output scales_t =
      output(Py_None, "scales_t", {q.scale_rows(K), blocks(M)}, q.scale, q.x, stream);
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_quantize_fp8_2d(q.x.t.const_data_ptr(), q.x.ld, M, K, q.block, fp8_code(q.type),
                             scale_code(q.scale), codes.t.data_ptr(), scales.t.data_ptr(),
                             codes_t.t.data_ptr(), scales_t.t.data_ptr(), stream.handle);
  Py_END_ALLOW_THREADS;
  return rc ? PyLong_FromLong(rc) : tuple_of({&codes, &scales, &codes_t, &scales_t});
  END_HANDLE_TH_ERRORS
}

// gemm_fp8(a, a_scales, b, b_scales, out_dtype, out, stream)
PyObject* gemm_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 7);
  const Codes x = codes_of(a[0], "a", true), w = codes_of(a[2], "b", false);
  const int64_t M = x.rows, K = x.cols, N = w.rows, KB = blocks(K);
  TORCH_CHECK_VALUE(w.cols == K, "b must have shape (N, ", K, "), got ",
                    shape_text(w.t.sizes()));
  const at::ScalarType scale = tensor(a[1], "a_scales").scalar_type();
  TORCH_CHECK_TYPE(scale == at::kByte || scale == at::kFloat,
                   "a_scales must be torch.uint8 or torch.float32, got ", dtype_name(scale));
  const at::Tensor& xs = checked(a[1], "a_scales", scale, {M, KB}, x.device);
  const int64_t rows = size_of(a[3], "b_scales", 2, 0);
  const bool by_rows = rows == N && rows != blocks(N);
  TORCH_CHECK_VALUE(!by_rows || scale == at::kByte,
                    "float32 b_scales must be those of 128 x 128 blocks, ",
                    shape_text({blocks(N), KB}));
  const at::Tensor& ws =
      checked(a[3], "b_scales", scale, {by_rows ? N : blocks(N), KB}, x.device);
  const at::ScalarType type = out_type(a[4], a[5]);
  const Stream stream = stream_of(a[6], x.device);
  Output y = output(a[5], "out", {M, N}, type, x, stream);
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_gemm_fp8(x.t.const_data_ptr(), fp8_code(x.type), xs.const_data_ptr(),
                      w.t.const_data_ptr(), ws.const_data_ptr(), scale_code(scale),
                      by_rows ? 1 : kFp8Block, M, N, K, out_code(type), y.t.data_ptr(),
                      stream.handle);
  Py_END_ALLOW_THREADS;
  return rc ? PyLong_FromLong(rc) : y.result();
  END_HANDLE_TH_ERRORS
}

// gemm_fp8_swiglu(a, a_scales, w13, w13_scales, want_act, want_gu, workspace,
//                 stream)
PyObject* gemm_fp8_swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 8);
  const Codes x = codes_of(a[0], "a", false), w = codes_of(a[2], "w13", false);
  const int64_t M = x.rows, K = x.cols, I = w.rows / 2, KB = blocks(K);
  TORCH_CHECK_VALUE(w.cols == K && I > 0 && w.rows % (2 * kFp8Block) == 0,
                    "w13 must be [2 I, ", K, "] with I a multiple of 128, got ",
                    shape_text(w.t.sizes()));
  const at::Tensor& xs = checked(a[1], "a_scales", at::kByte, {M, KB}, x.device);
  const at::Tensor& ws = checked(a[3], "w13_scales", at::kByte, {blocks(2 * I), KB}, x.device);
  const bool want_act = truth(a[4]), want_gu = truth(a[5]);
  int64_t bytes = 0;
  int rc = mxfp4_gemm_fp8_swiglu_workspace(M, I, K, &bytes);
  if (rc) return PyLong_FromLong(rc);
  const Stream stream = stream_of(a[7], x.device);
  Output codes = output(Py_None, "codes", {M, I}, at::kFloat8_e4m3fn, x, stream);
  Output scales = output(Py_None, "scales", {M, I / kFp8Block}, at::kByte, x, stream);
  Output act{at::Tensor(), nullptr}, gu{at::Tensor(), nullptr};
  if (want_act) act = output(Py_None, "act", {M, I}, at::kBFloat16, x, stream);
  if (want_gu) gu = output(Py_None, "gu", {M, 2 * I}, at::kBFloat16, x, stream);
  const Workspace space(a[6], bytes, x.device, stream);
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_gemm_fp8_swiglu(x.t.const_data_ptr(), xs.const_data_ptr(), w.t.const_data_ptr(),
                             ws.const_data_ptr(), M, I, K, codes.t.data_ptr(),
                             scales.t.data_ptr(), want_act ? act.t.data_ptr() : nullptr,
                             want_gu ? gu.t.data_ptr() : nullptr, space.ptr(), stream.handle);
  Py_END_ALLOW_THREADS;
  if (rc) return PyLong_FromLong(rc);
  if (want_act && want_gu) return tuple_of({&codes, &scales, &act, &gu});
  if (want_act) return tuple_of({&codes, &scales, &act});
  return want_gu ? tuple_of({&codes, &scales, &gu}) : tuple_of({&codes, &scales});
  END_HANDLE_TH_ERRORS
}

// swiglu_fp8_backward(dact, gu, dtype, stream)
PyObject* swiglu_fp8_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 4);
  const Rows d = rows_of(a[0], "dact");
  const int64_t M = d.rows, I = d.cols;
  TORCH_CHECK_VALUE(d.t.is_contiguous(), "dact must be contiguous (row-major)");
  TORCH_CHECK_VALUE(M > 0 && I > 0 && I % kFp8Block == 0,
                    "dact must be [M, I] with M > 0 and I a multiple of 128, got ",
                    shape_text(d.t.sizes()));
  const at::Tensor& gu = checked(a[1], "gu", at::kBFloat16, {M, 2 * I}, d.device);
  const at::ScalarType type = fp8_dtype(a[2]);
  const Stream stream = stream_of(a[3], d.device);
  Output codes = output(Py_None, "codes", {M, 2 * I}, type, d, stream);
  Output scales = output(Py_None, "scales", {M, 2 * I / kFp8Block}, at::kByte, d, stream);
  Output codes_t = output(Py_None, "codes_t", {2 * I, up16(M)}, type, d, stream);
  Output scales_t = output(Py_None, "scales_t", {2 * I, blocks(M)}, at::kByte, d, stream);
  int rc = 0;
  Py_BEGIN_ALLOW_THREADS;
  rc = mxfp4_swiglu_fp8_backward(d.t.const_data_ptr(), gu.const_data_ptr(), M, I, fp8_code(type),
                                 codes.t.data_ptr(), scales.t.data_ptr(), codes_t.t.data_ptr(),
                                 scales_t.t.data_ptr(), stream.handle);
  Py_END_ALLOW_THREADS;
  return rc ? PyLong_FromLong(rc) : tuple_of({&codes, &scales, &codes_t, &scales_t});
  END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"gemv", fast(gemv), METH_FASTCALL, nullptr},
    {"moe_route", fast(moe_route), METH_FASTCALL, nullptr},
    {"moe", fast(moe), METH_FASTCALL, nullptr},
    {"quantize_fp8", fast(quantize_fp8), METH_FASTCALL, nullptr},
    {"quantize_fp8_2d", fast(quantize_fp8_2d), METH_FASTCALL, nullptr},
    {"gemm_fp8", fast(gemm_fp8), METH_FASTCALL, nullptr},
    {"gemm_fp8_swiglu", fast(gemm_fp8_swiglu), METH_FASTCALL, nullptr},
    {"swiglu_fp8_backward", fast(swiglu_fp8_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
