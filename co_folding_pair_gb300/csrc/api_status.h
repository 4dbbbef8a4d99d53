// api_status.h -- how the C ABI's entry points report errors (internal).
#pragma once

#include <cuda_runtime.h>

#include "trimul.h"

namespace trimul {

// Sets this thread's message (trimul_last_error) and returns `s`.  Defined in trimul_api.cu.
trimul_status fail(trimul_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
trimul_status cuda_fail(cudaError_t e, const char* what);

}  // namespace trimul

#define TRY_CUDA(expr, what)                      \
  do {                                            \
    cudaError_t e_ = (expr);                      \
    if (e_ != cudaSuccess) return ::trimul::cuda_fail(e_, what); \
  } while (0)
