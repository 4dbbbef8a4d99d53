// step_ops.h -- launchers of the operators that end a training step, and of the
// linear layer in 8 bits (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "trimul.h"

namespace trimul {

// ---------------------------------------------------------------- AdamW
cudaError_t launch_adamw(const trimul_adamw_params& p, const trimul_adamw_tensor* t, const trimul_grad_tensor* g, int n, int32_t* count,
                         int num_sms, cudaStream_t s);

}  // namespace trimul
