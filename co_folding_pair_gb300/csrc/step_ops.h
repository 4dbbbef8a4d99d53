// step_ops.h -- the launcher of AdamW, which ends a training step (internal).
// Those of the linear layer in 8 bits are in linear8.h.
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
