// Host interface of the kernels around a projection: the residual norm
// (residual_norm.cu) and the low-rank adapters (lora.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

// Runs these kernels' bounded waits out on a barrier that never completes, with the
// given limit; one that answers anything else records tag + 1.
cudaError_t launch_selftest_block_waits(uint64_t timeout_ns, int tag, cudaStream_t stream);

// A checked residual-norm call (see nvfp4_residual_norm_args); rows > 0.
cudaError_t launch_residual_norm(const nvfp4_residual_norm_args &a, int num_sms,
                                 cudaStream_t stream);

// Bytes of workspace of launch_lora (0 where it needs none).
size_t lora_workspace_bytes(int64_t rows, int64_t k, int64_t n, int64_t rank);

// A checked adapter call (see nvfp4_lora_args); rows > 0.
cudaError_t launch_lora(const nvfp4_lora_args &p, cudaStream_t stream);

// The same for many rows, on 128-row tensor-core tiles (lora_tile.cu).  A tile
// whose rows have more than most_adapters different ones is left out, with a 1
// in its place of the array that *crowded receives (one int per tile, in the
// workspace).
size_t lora_tile_workspace_bytes(int64_t rows, int64_t rank);
cudaError_t launch_lora_tile(const nvfp4_lora_args &p, int most_adapters, const int **crowded,
                             cudaStream_t stream);

}  // namespace nvfp4
