// Argument checks and error reporting shared by the entry points that take no
// plan (embedding, expert products, gradient lists).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include <initializer_list>

#include "../../include/mg.h"

namespace mg {

struct OpPtr {
  const void* p;
  unsigned align;   // required alignment in bytes
};

// Sets the process-wide message and returns st.
mg_status op_fail(mg_status st, const char* fmt, ...);

// Before the launches of a call: every non-NULL pointer is aligned and is
// memory of the current device (a pointer of another device or of plain host
// memory is refused here, not left to fault on the device), and no CUDA error
// is pending on this thread.
mg_status op_begin(const char* fn, std::initializer_list<OpPtr> ptrs);

// The status of a call whose launches returned e.
mg_status op_end(const char* fn, cudaError_t e);

// Launch kern as a programmatic dependent of the kernel before it on s.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                             A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Multiprocessors of the current device.
int device_sms();

}  // namespace mg
