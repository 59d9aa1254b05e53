// Host interface of the kernels around a projection: the residual norm
// (residual_norm.cu) and the low-rank adapters (lora.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

// A checked residual-norm call (see nvfp4_residual_norm_args); rows > 0.
cudaError_t launch_residual_norm(const nvfp4_residual_norm_args &a, int num_sms,
                                 cudaStream_t stream);

}  // namespace nvfp4
