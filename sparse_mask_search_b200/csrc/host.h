// Host-side helpers shared by the translation units of the C ABI.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/tsenor.h"

namespace tsenor {

// Records the message tsenor_last_error returns; the status is TSENOR_ERR_CUDA.
tsenor_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Adds the rows that failed in the distillation kernels on the current device
// since the last call to *count and resets them (ordered on `st`).
cudaError_t read_row_failures(cudaStream_t st, unsigned long long* count);
// The same for the threads of tsenor_matmul's kernels whose bounded wait ran out.
cudaError_t read_stalled(cudaStream_t st, unsigned long long* count);

}  // namespace tsenor
