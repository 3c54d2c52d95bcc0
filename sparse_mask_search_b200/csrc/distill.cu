// Distillation from a teacher's top logits, forward and backward.
//
// Row (token) with student logits z, temperature T, teacher entries (i_j, t_j):
//   p_j = exp(t_j / T - c),  c = logsumexp_j(t_j / T) or the teacher's own normaliser
//   q = softmax(z / T),  lse = logsumexp(z / T)
//   loss = T^2 sum_j p_j (log p_j - log q_{i_j})
//   dz_v = w T (P q_v - sum_{j: i_j = v} p_j),  P = sum_j p_j
// One pass keeps the running maximum and sum of the softmax (fp32); the
// gradient follows from z and lse alone.
#include <type_traits>

#include "common.cuh"
#include "host.h"

namespace tsenor {
namespace {

__device__ unsigned long long g_row_failures;

constexpr int kThreads = 512;
constexpr int kMaxTop = TSENOR_DISTILL_MAX_TOP;
constexpr float kLog2E = 1.4426950408889634f;

enum Mode { kLoss, kStep, kGrad };

struct DistillArgs {
    const void* logits;
    int64_t rows, vocab, ld;
    const int32_t* index;
    const float* top_logits;
    int top;
    const float* teacher_lse;
    float temperature;
    const float* weight;
    float* loss;
    float* lse;
    void* grad;
    int64_t ldg;
};

template <typename T>
__device__ __forceinline__ float read(const typename T::storage* p) {
    if constexpr (std::is_same<T, BF16>::value) return __uint_as_float(uint32_t(*p) << 16);
    else return *p;
}
template <typename T>
__device__ __forceinline__ void write(typename T::storage* p, float x) {
    if constexpr (std::is_same<T, BF16>::value) {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
        *p = h;
    } else {
        *p = x;
    }
}

__device__ float block_max(float v, float* red) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, s));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int k = 1; k < kThreads / 32; ++k) v = fmaxf(v, red[k]);
    __syncthreads();
    return v;
}
__device__ float block_sum(float v, float* red) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v += __shfl_xor_sync(kFullMask, v, s);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int k = 1; k < kThreads / 32; ++k) v += red[k];
    __syncthreads();
    return v;
}

template <typename T, Mode MODE>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
    __shared__ float red[kThreads / 32];
    __shared__ int idx[kMaxTop];
    __shared__ float p[kMaxTop], zt[kMaxTop];
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const auto* z = static_cast<const typename T::storage*>(a.logits) + row * a.ld;
    const float inv_t = 1.f / a.temperature;
    bool bad = false;
    // the teacher's entries and their weights
    float high = -INFINITY;
    for (int j = t; j < a.top; j += kThreads) {
        const int i = a.index[row * a.top + j];
        const float v = a.top_logits[row * a.top + j] / a.temperature;
        bad = bad || i >= a.vocab || (i >= 0 && !(v < INFINITY));
        idx[j] = i >= 0 && i < a.vocab ? i : -1;
        p[j] = i >= 0 && i < a.vocab ? v : -INFINITY;
        zt[j] = i >= 0 && i < a.vocab ? read<T>(z + i) : 0.f;
        high = fmaxf(high, p[j]);
    }
    high = block_max(high, red);
    const bool empty = high == -INFINITY;
    float c = 0.f;
    if (!empty) {
        if (a.teacher_lse) {
            c = a.teacher_lse[row];
            bad = bad || !(fabsf(c) < INFINITY);
        } else {
            float s = 0.f;
            for (int j = t; j < a.top; j += kThreads) s += expf(p[j] - high);
            c = high + logf(block_sum(s, red));
        }
    }
    // the student's normaliser
    float lse;
    if constexpr (MODE == kGrad) {
        lse = a.lse[row];
    } else {
        float m = -INFINITY, s = 0.f;
        bool nan = false;
        for (int64_t v = t; v < a.vocab; v += kThreads) {
            const float x = read<T>(z + v);
            nan = nan || !(x < INFINITY);
            m = fmaxf(m, x);
        }
        m = block_max(m, red);
        if (m > -INFINITY)
            for (int64_t v = t; v < a.vocab; v += kThreads) s += ex2((read<T>(z + v) - m) * (inv_t * kLog2E));
        if (nan) s = NAN;
        s = block_sum(s, red);
        lse = m == -INFINITY ? m : m / a.temperature + logf(s);
    }
    bad = bad || (!empty && !(fabsf(lse) < INFINITY));
    bad = __syncthreads_or(bad);
    float part = 0.f, total = 0.f;
    for (int j = t; j < a.top; j += kThreads) {
        const float logp = p[j] - c, w = empty ? 0.f : expf(logp);
        if (w > 0.f) part += w * (logp - (zt[j] / a.temperature - lse));
        total += w;
        p[j] = w;
    }
    total = block_sum(total, red);
    if constexpr (MODE != kGrad) {
        part = block_sum(part, red);
        if (t == 0) a.loss[row] = bad ? NAN : empty ? 0.f : a.temperature * a.temperature * part;
    }
    if (MODE == kLoss && t == 0) a.lse[row] = bad ? NAN : lse;
    if (bad && t == 0) atomicAdd(&g_row_failures, 1ull);
    if constexpr (MODE != kLoss) {
        auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
        const float by = a.temperature * (a.weight ? a.weight[row] : 1.f);
        if (bad || empty || by == 0.f) {
            for (int64_t v = t; v < a.vocab; v += kThreads) write<T>(g + v, 0.f);
            return;
        }
        const float scale = by * total;
        for (int64_t v = t; v < a.vocab; v += kThreads)
            write<T>(g + v, scale * ex2(fmaf(read<T>(z + v), inv_t, -lse) * kLog2E));
        __syncthreads();
        // the teacher's entries: the first one of an index writes for all of its kind, in order
        for (int j = t; j < a.top; j += kThreads) {
            if (idx[j] < 0) continue;
            bool first = true;
            float w = 0.f;
            for (int k = 0; k < a.top; ++k)
                if (idx[k] == idx[j]) {
                    first = first && k >= j;
                    w += p[k];
                }
            if (first) write<T>(g + idx[j], scale * ex2(fmaf(zt[j], inv_t, -lse) * kLog2E) - by * w);
        }
    }
}

template <Mode MODE>
tsenor_status run_distill(tsenor_dtype dtype, const DistillArgs& a, cudaStream_t st, const char* what) {
    if (dtype == TSENOR_BF16) distill_kernel<BF16, MODE><<<unsigned(a.rows), kThreads, 0, st>>>(a);
    else distill_kernel<F32, MODE><<<unsigned(a.rows), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, what);
}

tsenor_status check_distill(int dtype, const DistillArgs& a) {
    if (dtype != TSENOR_F32 && dtype != TSENOR_BF16) return TSENOR_ERR_ARG;
    if (a.rows < 0 || a.rows > (int64_t(1) << 31) - 1 || a.vocab < 1 || a.vocab > TSENOR_DISTILL_MAX_VOCAB ||
        a.top < 0 || a.top > kMaxTop)
        return TSENOR_ERR_SHAPE;
    if (!(a.temperature > 0.f) || a.temperature > 3.0e38f || a.temperature < 1.0e-6f) return TSENOR_ERR_ARG;
    if (a.rows == 0) return TSENOR_OK;
    if (!a.logits || !aligned(a.logits, dtype == TSENOR_BF16 ? 2 : 4) || a.ld < a.vocab) return TSENOR_ERR_ARG;
    if (a.top > 0 && (!a.index || !aligned(a.index, 4) || !a.top_logits || !aligned(a.top_logits, 4)))
        return TSENOR_ERR_ARG;
    if (!aligned(a.teacher_lse, 4) || !aligned(a.weight, 4)) return TSENOR_ERR_ARG;
    return TSENOR_OK;
}

bool grad_ok(int dtype, const DistillArgs& a) {
    // in place means the same rows: any other overlap would overwrite logits not yet read
    return a.grad && aligned(a.grad, dtype == TSENOR_BF16 ? 2 : 4) && a.ldg >= a.vocab &&
           (a.grad != a.logits || a.ldg == a.ld);
}

}  // namespace

cudaError_t read_row_failures(cudaStream_t st, unsigned long long* count) {
    unsigned long long v = 0;
    const unsigned long long zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_row_failures, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemcpyToSymbolAsync(g_row_failures, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess) *count += v;
    return e;
}

}  // namespace tsenor

using namespace tsenor;

extern "C" tsenor_status tsenor_distill_loss(const void* logits, tsenor_dtype dtype, int64_t rows, int64_t vocab,
                                             int64_t ld, const int32_t* index, const float* top_logits, int top,
                                             const float* teacher_lse, float temperature, float* loss, float* lse,
                                             tsenor_stream_t stream) {
    const DistillArgs a{logits, rows, vocab, ld, index, top_logits, top, teacher_lse, temperature, nullptr, loss, lse,
                        nullptr, 0};
    const tsenor_status s = check_distill(dtype, a);
    if (s != TSENOR_OK || rows == 0) return s;
    if (!loss || !aligned(loss, 4) || !lse || !aligned(lse, 4)) return TSENOR_ERR_ARG;
    return run_distill<kLoss>(dtype, a, (cudaStream_t)stream, "tsenor_distill_loss launch");
}

extern "C" tsenor_status tsenor_distill_step(const void* logits, tsenor_dtype dtype, int64_t rows, int64_t vocab,
                                             int64_t ld, const int32_t* index, const float* top_logits, int top,
                                             const float* teacher_lse, float temperature, const float* weight,
                                             float* loss, void* grad, int64_t ldg, tsenor_stream_t stream) {
    const DistillArgs a{logits, rows, vocab, ld, index, top_logits, top, teacher_lse, temperature, weight, loss,
                        nullptr, grad, ldg};
    const tsenor_status s = check_distill(dtype, a);
    if (s != TSENOR_OK || rows == 0) return s;
    if (!loss || !aligned(loss, 4) || !grad_ok(dtype, a)) return TSENOR_ERR_ARG;
    return run_distill<kStep>(dtype, a, (cudaStream_t)stream, "tsenor_distill_step launch");
}

extern "C" tsenor_status tsenor_distill_grad(const void* logits, tsenor_dtype dtype, int64_t rows, int64_t vocab,
                                             int64_t ld, const int32_t* index, const float* top_logits, int top,
                                             const float* teacher_lse, float temperature, const float* lse,
                                             const float* weight, void* grad, int64_t ldg, tsenor_stream_t stream) {
    const DistillArgs a{logits, rows, vocab, ld, index, top_logits, top, teacher_lse, temperature, weight, nullptr,
                        const_cast<float*>(lse), grad, ldg};
    const tsenor_status s = check_distill(dtype, a);
    if (s != TSENOR_OK || rows == 0) return s;
    if (!lse || !aligned(lse, 4) || !grad_ok(dtype, a)) return TSENOR_ERR_ARG;
    return run_distill<kGrad>(dtype, a, (cudaStream_t)stream, "tsenor_distill_grad launch");
}
