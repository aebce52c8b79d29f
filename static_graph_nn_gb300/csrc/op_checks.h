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

// Multiprocessors of the current device.
int device_sms();

}  // namespace mg
