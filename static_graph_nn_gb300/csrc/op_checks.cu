#include "op_checks.h"

#include <stdint.h>

#include <cstdarg>
#include <cstdio>

#include "kernels.h"

namespace mg {

mg_status op_fail(mg_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_global_error(buf);
  return st;
}

mg_status op_begin(const char* fn, std::initializer_list<OpPtr> ptrs) {
  for (const OpPtr& q : ptrs)
    if (q.p && reinterpret_cast<uintptr_t>(q.p) % q.align)
      return op_fail(MG_ERR_ALIGN, "%s: pointers must be %u-byte aligned", fn, q.align);
  cudaError_t e = cudaPeekAtLastError();
  if (e != cudaSuccess)
    return op_fail(MG_ERR_CUDA, "%s: a CUDA error was already pending before the call (%s); nothing launched",
                   fn, cudaGetErrorString(e));
  int dev = -1;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return op_fail(MG_ERR_CUDA, "%s: no usable current CUDA device (%s)", fn, cudaGetErrorString(e));
  }
  for (const OpPtr& q : ptrs) {
    if (!q.p) continue;
    cudaPointerAttributes a;
    e = cudaPointerGetAttributes(&a, q.p);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return op_fail(MG_ERR_CUDA, "%s: cudaPointerGetAttributes: %s", fn, cudaGetErrorString(e));
    }
    if (a.type == cudaMemoryTypeUnregistered)
      return op_fail(MG_ERR_INVALID_ARG, "%s: a pointer is not device memory", fn);
    if (a.type == cudaMemoryTypeDevice && a.device != dev)
      return op_fail(MG_ERR_INVALID_ARG, "%s: a pointer belongs to device %d but device %d is current", fn,
                     a.device, dev);
  }
  return MG_OK;
}

mg_status op_end(const char* fn, cudaError_t e) {
  if (e == cudaSuccess) return MG_OK;
  cudaGetLastError();
  return op_fail(MG_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = 148;
  }
  return n;
}

}  // namespace mg
