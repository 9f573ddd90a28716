/* A HIP runtime that launches nothing: a gfx950 device is current, launches
 * are counted, and a launch that asks for more dynamic LDS than its kernel's
 * limit fails. Loaded before libmxfp4.so with its symbols global, it takes the
 * place of the calls that the library's host code makes. */
#define __HIP_PLATFORM_AMD__ 1
#include <hip/hip_runtime_api.h>
#include <string.h>

enum { kKernels = 256 };
static const void* kernels[kKernels];
static size_t limits[kKernels];
static hipError_t last = hipSuccess;
static int inside = 0;

int fake_launches = 0;
size_t fake_most_lds = 0;
void (*fake_between)(void) = 0; /* another thread's call, between a set and what follows */

static size_t* limit_of(const void* f) {
  int i = 0;
  while (i < kKernels - 1 && kernels[i] && kernels[i] != f) ++i;
  if (!kernels[i]) {
    kernels[i] = f;
    limits[i] = 65536;
  }
  return &limits[i];
}

hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}

hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int dev) {
  (void)dev;
  memset(p, 0, sizeof *p);
  strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}

hipError_t hipDeviceGetAttribute(int* value, hipDeviceAttribute_t attr, int dev) {
  (void)attr;
  (void)dev;
  *value = 256;
  return hipSuccess;
}

hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute attr, int value) {
  if (attr != hipFuncAttributeMaxDynamicSharedMemorySize) return hipErrorInvalidValue;
  *limit_of(f) = (size_t)value;
  if (fake_between && !inside) {
    inside = 1;
    fake_between();
    inside = 0;
  }
  return hipSuccess;
}

static dim3 next_grid, next_block;
static size_t next_lds;
static hipStream_t next_stream;

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  next_grid = grid;
  next_block = block;
  next_lds = lds;
  next_stream = stream;
  return hipSuccess;
}

hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = next_grid;
  *block = next_block;
  *lds = next_lds;
  *stream = next_stream;
  return hipSuccess;
}

hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t lds,
                           hipStream_t stream) {
  (void)args;
  (void)stream;
  ++fake_launches;
  if (lds > fake_most_lds) fake_most_lds = lds;
  if (lds > *limit_of(f) || lds > 163840 || block.x > 1024 || grid.y > 65535 || grid.z > 65535 ||
      (unsigned long long)grid.x * block.x >= 1ull << 32)
    last = hipErrorInvalidConfiguration;
  return last;
}

hipError_t hipGetLastError(void) {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}
