// Beside matmul.cu and distill.cu (sparse_mask_search_b200/csrc) in a library for tests, whose limited waits run out
// as the tests ask (TSENOR_GIVE_UP): what those files take from others, and their counters.
#include "../sparse_mask_search_b200/csrc/host.h"

namespace tsenor {
tsenor_status cuda_fail(cudaError_t, const char*) { return TSENOR_ERR_CUDA; }
}  // namespace tsenor

// How many warps gave up (and rows failed) since the last call; -1 for an error of CUDA.
extern "C" long long give_up_count() {
    unsigned long long* at[2];
    if (tsenor::stalls(&at[0]) != cudaSuccess || tsenor::row_failures(&at[1]) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return -1;
    long long sum = 0;
    for (auto* p : at) {
        unsigned long long v = 0;
        if (cudaMemcpy(&v, p, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess || cudaMemset(p, 0, sizeof(v)) != cudaSuccess) return -1;
        sum += (long long)v;
    }
    return sum;
}
