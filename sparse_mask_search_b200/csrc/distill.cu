// Distillation from a teacher's top logits, forward and backward.
//
// Row (token) with student logits z, temperature T, teacher entries (i_j, t_j):
//   p_j = exp(t_j / T - c),  c = logsumexp_j(t_j / T) or the teacher's own normaliser
//   q = softmax(z / T),  lse = logsumexp(z / T)
//   loss = T^2 sum_j p_j (log p_j - log q_{i_j})
//   dz_v = w T (P q_v - sum_{j: i_j = v} p_j),  P = sum_j p_j
//
// Bound by memory: z is read once and dz written once.  For the loss, a row is
// cut into slices of at most 64 KB, one to a CTA of a cluster of up to 8; bulk
// copies bring the slice into shared memory, where its maximum, its sum of
// exponentials and, for the step, its gradient are taken, and the CTAs exchange one
// (maximum, sum, loss term) each.  Three CTAs to an SM overlap one row's loads with
// another's arithmetic and stores.  A few rows get more and smaller slices.  The
// gradient alone needs nothing but z and lse: it streams through registers.
// Sums are fp32, the few scalars of a row fp64.
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "tensor.h"

namespace tsenor {
namespace {

__device__ unsigned long long g_row_failures;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = TSENOR_DISTILL_MAX_TOP;
constexpr int kSegments = 4;                     // of a slice's copy, each with its own barrier
constexpr int kMaxSlices = 8;
constexpr int kSliceBytes = 64 * 1024;
constexpr float kLog2E = 1.4426950408889634f;

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

__device__ __forceinline__ uint16_t round_bf16(float x) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
}
template <typename T>
__device__ __forceinline__ float read(const typename T::storage* p) {
    if constexpr (std::is_same<T, BF16>::value) return __uint_as_float(uint32_t(*p) << 16);
    else return *p;
}
template <typename T>
__device__ __forceinline__ void write(typename T::storage* p, float x) {
    if constexpr (std::is_same<T, BF16>::value) *p = round_bf16(x);
    else *p = x;
}
// Entries 2i and 2i + 1 of a 16-byte chunk (bf16: i < 4, fp32: i < 2), and back.
template <typename T>
__device__ __forceinline__ float2 pair_of(const uint4& v, int i) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (std::is_same<T, BF16>::value)
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else
        return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}
template <typename T>
__device__ __forceinline__ void set_pair(uint32_t (&w)[4], int i, float2 x) {
    if constexpr (std::is_same<T, BF16>::value)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x.y), "f"(x.x));
    else {
        w[2 * i] = __float_as_uint(x.x);
        w[2 * i + 1] = __float_as_uint(x.y);
    }
}

struct Max {
    __device__ static float of(float a, float b) { return fmaxf(a, b); }
};
struct Sum {
    template <typename X>
    __device__ static X of(X a, X b) { return a + b; }
};
// Over the block, in a fixed order; the result in every thread.
template <typename Op, typename X>
__device__ X reduce(X v, X* red) {
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) v = Op::of(v, __shfl_xor_sync(kFullMask, v, s));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) v = Op::of(v, red[k]);
    __syncthreads();
    return v;
}

// A row's columns in memory: `head` entries up to the first 16-byte boundary, `chunks` of 16
// bytes, `tail` entries.  Slice r of n has a share of the chunks; the first also
// has the head, the last the tail.
template <typename T>
struct Slice {
    static constexpr int kPer = 16 / sizeof(typename T::storage);
    int head, tail, chunk0, chunks;              // of this slice
    int first;                                   // column of its first chunk
    int vocab;

    __device__ Slice(const typename T::storage* z, int vocab_, int r, int n) : vocab(vocab_) {
        int h = int(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(typename T::storage));
        if (h > vocab) h = vocab;
        const int all = (vocab - h) / kPer;
        chunk0 = int(int64_t(all) * r / n);
        chunks = int(int64_t(all) * (r + 1) / n) - chunk0;
        head = r == 0 ? h : 0;
        tail = r == n - 1 ? vocab - h - all * kPer : 0;
        first = h + chunk0 * kPer;
    }
    __device__ int extras() const { return head + tail; }              // fewer than 2 * kPer
    __device__ int extra(int i) const { return i < head ? i : vocab - tail + i - head; }     // their columns
    __device__ bool has(int v) const {
        return (v >= first && v < first + chunks * kPer) || v < head || (v >= vocab - tail && v < vocab);
    }
};

// The teacher's entries of a row in shared memory, their number rounded up to 4.
struct Teacher {
    float* p;
    int* index;                                  // 16-byte aligned; -1: no entry
    float* target;                               // grad_kernel: the gradient of the entry's column

    __device__ Teacher(void* at, int top) : p(static_cast<float*>(at)) {
        index = reinterpret_cast<int*>(p + (top + 3) / 4 * 4);
        target = reinterpret_cast<float*>(index + (top + 3) / 4 * 4);
    }
};

// Fills idx and p; returns P = sum p.  `empty`: no entry has weight; `bad`: the row fails.
__device__ float teacher_weights(const DistillArgs& a, int64_t row, const Teacher& s, float* red, bool* empty, bool* bad) {
    bool wrong = false;
    float high = -INFINITY;
    for (int j = threadIdx.x; j < (a.top + 3) / 4 * 4; j += kThreads) {
        const int i = j < a.top ? a.index[row * a.top + j] : -1;
        const float v = j < a.top ? a.top_logits[row * a.top + j] / a.temperature : 0.f;
        wrong = wrong || i >= a.vocab || (i >= 0 && !(v < INFINITY));
        const bool in = i >= 0 && i < a.vocab;
        s.index[j] = in ? i : -1;
        s.p[j] = in ? v : -INFINITY;
        high = fmaxf(high, s.p[j]);
    }
    high = reduce<Max>(high, red);
    *empty = high == -INFINITY;
    float c = 0.f;
    if (!*empty) {
        if (a.teacher_lse) {
            c = a.teacher_lse[row];
            wrong = wrong || !(fabsf(c) < INFINITY);
        } else {
            float sum = 0.f;
            for (int j = threadIdx.x; j < a.top; j += kThreads) sum += expf(s.p[j] - high);
            c = high + logf(reduce<Sum>(sum, red));
        }
    }
    float total = 0.f;
    for (int j = threadIdx.x; j < a.top; j += kThreads) {
        const float w = *empty ? 0.f : expf(s.p[j] - c);
        s.p[j] = w;
        total += w;
    }
    *bad = __syncthreads_or(wrong);
    return reduce<Sum>(total, red);
}

// Calls f(j, v, sum of the weights of index v) for the entries of a slice, each index once.
template <typename T, typename F>
__device__ __forceinline__ void each_target(const Teacher& s, int top, const Slice<T>& slice, F f) {
    for (int j = threadIdx.x; j < top; j += kThreads) {
        const int v = s.index[j];
        if (v < 0 || !slice.has(v)) continue;
        bool first = true;
        float w = 0.f;
        for (int k = 0; k < top; k += 4) {
            const int4 o = *reinterpret_cast<const int4*>(s.index + k);
            if (o.x == v) { first = first && k >= j; w += s.p[k]; }
            if (o.y == v) { first = first && k + 1 >= j; w += s.p[k + 1]; }
            if (o.z == v) { first = first && k + 2 >= j; w += s.p[k + 2]; }
            if (o.w == v) { first = first && k + 3 >= j; w += s.p[k + 3]; }
        }
        if (first) f(j, v, w);
    }
}

// Gradient 0 for the columns of a slice.
template <typename T>
__device__ void write_zeros(typename T::storage* g, const Slice<T>& slice, bool vec) {
    if (vec) {
        uint4* o = reinterpret_cast<uint4*>(g + slice.first);
        for (int i = threadIdx.x; i < slice.chunks; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    } else {
        for (int i = threadIdx.x; i < slice.chunks * Slice<T>::kPer; i += kThreads) write<T>(g + slice.first + i, 0.f);
    }
    for (int i = threadIdx.x; i < slice.extras(); i += kThreads) write<T>(g + slice.extra(i), 0.f);
}

// One chunk of gradient from f(logit) of its entries.
template <typename T, typename F>
__device__ __forceinline__ void write_chunk(typename T::storage* g, const uint4& z, bool vec, F f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < Slice<T>::kPer / 2; ++i) set_pair<T>(w, i, f(pair_of<T>(z, i)));
    if (vec) {
        *reinterpret_cast<uint4*>(g) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < Slice<T>::kPer; ++k) {
            if constexpr (std::is_same<T, BF16>::value) g[k] = uint16_t(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
            else g[k] = __uint_as_float(w[k]);
        }
    }
}

// What a slice tells the others of its row.
struct Share {
    float high, sum;
    double term;
};

// Loss (STEP: and gradient).  A cluster of `slices` CTAs to a row.
template <typename T, bool STEP>
__global__ void __launch_bounds__(kThreads) loss_kernel(const DistillArgs a, const int slices, const int chunk_room) {
    extern __shared__ __align__(128) uint4 chunk[];
    __shared__ float red[kWarps];
    __shared__ double red64[kWarps];
    __shared__ Share share[kMaxSlices];
    __shared__ float extra[2 * Slice<T>::kPer];
    __shared__ float row_high, row_sum;
    __shared__ uint64_t bar[kSegments];
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x / slices;
    const int rank = slices > 1 ? int(cluster_rank()) : 0;
    const auto* z = static_cast<const typename T::storage*>(a.logits) + row * a.ld;
    auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
    const Slice<T> slice(z, int(a.vocab), rank, slices);
    const Teacher teacher(chunk + chunk_room, a.top);
    const bool vec = STEP && ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    if (slices > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");      // every CTA of the row has begun

    auto start_copy = [&] {                      // one thread; segment i has chunks [chunks i / kSegments, ...)
        for (int i = 0; i < kSegments; ++i) mbar_init(bar + i, 1);
        mbar_init_fence();
        for (int i = 0; i < kSegments; ++i) {
            const int c0 = slice.chunks * i / kSegments, n = slice.chunks * (i + 1) / kSegments - c0;
            mbar_arrive_expect_tx(bar + i, n * 16);
            if (n > 0) bulk_load(chunk + c0, z + slice.first + c0 * Slice<T>::kPer, n * 16, bar + i);
        }
    };
    if (!STEP && t == 0) start_copy();
    if (t < slice.extras()) extra[t] = read<T>(z + slice.extra(t));
    bool empty, bad;
    const float total = teacher_weights(a, row, teacher, red, &empty, &bad);
    if (STEP && (empty || bad)) {                // the logits are not read
        if (slices > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        write_zeros<T>(g, slice, vec);
        if (t == 0 && rank == 0) {
            a.loss[row] = bad ? NAN : 0.f;
            if (bad) atomicAdd(&g_row_failures, 1ull);
        }
        return;
    }
    if (STEP && t == 0) start_copy();
    if (STEP) __syncthreads();

    const float inv_t = 1.f / a.temperature, scale2 = inv_t * kLog2E;
    float high = -INFINITY;
    bool stalled = false;
    for (int i = 0; i < kSegments; ++i) {
        if (!mbar_wait_bounded(bar + i, 0)) stalled = true;
        const int c1 = slice.chunks * (i + 1) / kSegments;
        for (int c = slice.chunks * i / kSegments + t; c < c1; c += kThreads) {
            const uint4 v = chunk[c];
            if constexpr (std::is_same<T, BF16>::value) {
                uint32_t m, n;
                asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
                asm("max.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(v.z), "r"(v.w));
                asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
                high = fmaxf(high, fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u)));
            } else {
                high = fmaxf(high, fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                                         fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))));
            }
        }
    }
    if (t < slice.extras()) high = fmaxf(high, extra[t]);
    high = reduce<Max>(high, red);
    // a NaN or +inf anywhere makes the sum NaN
    const float base = high == -INFINITY ? 0.f : high;
    const float2 minus = make_float2(-base, -base), by2 = make_float2(scale2, scale2);
    float2 sum2 = make_float2(0.f, 0.f);
    for (int c = t; c < slice.chunks; c += kThreads) {
        const uint4 v = chunk[c];
#pragma unroll
        for (int i = 0; i < Slice<T>::kPer / 2; ++i) {
            const float2 x = mul2(add2(pair_of<T>(v, i), minus), by2);
            sum2 = add2(sum2, make_float2(ex2(x.x), ex2(x.y)));
        }
    }
    float sum = sum2.x + sum2.y;
    if (t < slice.extras()) sum += ex2((extra[t] - base) * scale2);
    if (stalled) sum = NAN;
    sum = reduce<Sum>(sum, red);

    // sum_j p_j (log p_j - z_j / T) of the entries in this slice; their logits replace nothing yet
    auto logit_at = [&](int v) {
        if (v < slice.head) return extra[v];
        if (v >= slice.first && v < slice.first + slice.chunks * Slice<T>::kPer)
            return read<T>(reinterpret_cast<const typename T::storage*>(chunk) + (v - slice.first));
        return extra[slice.head + v - (slice.vocab - slice.tail)];
    };
    double term = 0.0;
    for (int j = t; j < a.top; j += kThreads) {
        const int v = teacher.index[j];
        const float w = teacher.p[j];
        if (v >= 0 && w > 0.f && slice.has(v))
            term += double(w) * (log(double(w)) - double(logit_at(v)) / double(a.temperature));
    }
    term = reduce<Sum>(term, red64);
    if (slices > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (t < slices) {
            const uint32_t to = cluster_addr(smem_u32(share + rank), t);
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(high), "f"(sum) : "memory");
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to + 8), "d"(term) : "memory");
        }
        cluster_sync();
    } else if (t == 0) {
        share[0] = Share{high, sum, term};
    }
    if (t == 0) {
        float m = share[0].high;
        for (int k = 1; k < slices; ++k) m = fmaxf(m, share[k].high);
        float s = 0.f;
        double all = 0.0;
        for (int k = 0; k < slices; ++k) {
            // a slice without a finite logit adds nothing, but a NaN
            s += share[k].high == -INFINITY ? share[k].sum : share[k].sum * ex2((share[k].high - m) * scale2);
            all += share[k].term;
        }
        const double lse = m == -INFINITY ? double(m) : double(m) / double(a.temperature) + log(double(s));
        const bool failed = bad || (!empty && !(fabs(lse) < double(INFINITY)));
        if (rank == 0) {
            a.loss[row] = failed ? NAN : empty ? 0.f
                          : float(double(a.temperature) * double(a.temperature) * (all + double(total) * lse));
            if (!STEP) a.lse[row] = failed ? NAN : float(lse);
            if (failed) atomicAdd(&g_row_failures, 1ull);
        }
        row_high = m;
        row_sum = failed ? 0.f : s;
    }
    if constexpr (STEP) {
        __syncthreads();
        const float by = a.temperature * (a.weight ? a.weight[row] : 1.f);
        if (row_sum == 0.f || by == 0.f) {
            write_zeros<T>(g, slice, vec);
            return;
        }
        const float scale = by * total / row_sum, m = row_high;
        auto at = [&](float x) { return scale * ex2((x - m) * scale2); };
        const float2 minus_m = make_float2(-m, -m), scale_2 = make_float2(scale, scale);
        for (int c = t; c < slice.chunks; c += kThreads)
            write_chunk<T>(g + slice.first + c * Slice<T>::kPer, chunk[c], vec, [&](float2 x) {
                x = mul2(add2(x, minus_m), by2);
                return mul2(make_float2(ex2(x.x), ex2(x.y)), scale_2);
            });
        if (t < slice.extras()) write<T>(g + slice.extra(t), at(extra[t]));
        __syncthreads();                         // the entries' columns are written again
        each_target<T>(teacher, a.top, slice, [&](int, int v, float w) { write<T>(g + v, at(logit_at(v)) - by * w); });
    }
}

// The gradient from lse; blockIdx.x is a row's slice.
template <typename T>
__global__ void __launch_bounds__(kThreads) grad_kernel(const DistillArgs a, const int slices) {
    extern __shared__ __align__(128) uint4 chunk[];
    __shared__ float red[kWarps];
    const Teacher teacher(chunk, a.top);
    constexpr int kAhead = 4;                    // chunks of a thread in flight
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x / slices;
    const int rank = int(blockIdx.x % slices);
    const auto* z = static_cast<const typename T::storage*>(a.logits) + row * a.ld;
    auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
    const Slice<T> slice(z, int(a.vocab), rank, slices);
    const bool vec = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    bool empty, bad;
    const float total = teacher_weights(a, row, teacher, red, &empty, &bad);
    const float lse = a.lse[row];
    const float by = a.temperature * (a.weight ? a.weight[row] : 1.f);
    bad = bad || (!empty && !(fabsf(lse) < INFINITY));
    if (bad && rank == 0 && t == 0) atomicAdd(&g_row_failures, 1ull);
    if (bad || empty || by == 0.f) {
        write_zeros<T>(g, slice, vec);
        return;
    }
    const float inv_t = 1.f / a.temperature, scale = by * total;
    auto at = [&](float x) { return scale * ex2(fmaf(x, inv_t, -lse) * kLog2E); };
    // the entries' gradients before anything is written: grad may be the logits
    each_target<T>(teacher, a.top, slice, [&](int j, int v, float w) { teacher.target[j] = at(read<T>(z + v)) - by * w; });
    __syncthreads();
    const uint4* in = reinterpret_cast<const uint4*>(z + slice.first);
    const float2 inv2 = make_float2(inv_t, inv_t), minus = make_float2(-lse, -lse), l2 = make_float2(kLog2E, kLog2E),
                 scale_2 = make_float2(scale, scale);
    for (int c = t; c < slice.chunks; c += kAhead * kThreads) {
        uint4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c + i * kThreads < slice.chunks) v[i] = in[c + i * kThreads];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c + i * kThreads < slice.chunks)
                write_chunk<T>(g + slice.first + (c + i * kThreads) * Slice<T>::kPer, v[i], vec, [&](float2 x) {
                    x = mul2(fma2(x, inv2, minus), l2);
                    return mul2(make_float2(ex2(x.x), ex2(x.y)), scale_2);
                });
    }
    if (t < slice.extras()) write<T>(g + slice.extra(t), at(read<T>(z + slice.extra(t))));
    __syncthreads();
    each_target<T>(teacher, a.top, slice, [&](int j, int v, float) { write<T>(g + v, teacher.target[j]); });
}

// Slices of a row: at most kSliceBytes each, and for few rows enough CTAs to fill the
// device twice, of 4 KB at least.
int slices_of(int64_t rows, int64_t row_bytes) {
    int n = 1;
    while (n < kMaxSlices && (row_bytes > int64_t(n) * kSliceBytes || (rows * n < 296 && row_bytes > int64_t(n) * 8192))) n *= 2;
    return n;
}

template <typename T, bool STEP>
cudaError_t launch_loss(const DistillArgs& a, cudaStream_t st) {
    const int64_t row_bytes = a.vocab * int64_t(sizeof(typename T::storage));
    const int slices = slices_of(a.rows, row_bytes);
    const int chunk_room = int((row_bytes / 16 + slices - 1) / slices);
    const unsigned bytes = unsigned(chunk_room * 16 + (a.top + 3) / 4 * 4 * 8);
    cudaError_t e = cudaFuncSetAttribute(loss_kernel<T, STEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows * slices));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(slices);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = slices > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, loss_kernel<T, STEP>, a, slices, chunk_room);
}

template <typename T>
cudaError_t launch_grad(const DistillArgs& a, cudaStream_t st) {
    // about 64 KB to a CTA: the teacher's weights are computed for each
    const int64_t row_bytes = a.vocab * int64_t(sizeof(typename T::storage));
    const int slices = a.rows >= 296 ? int((row_bytes + kSliceBytes - 1) / kSliceBytes)
                                     : int((row_bytes + kSliceBytes / 8 - 1) / (kSliceBytes / 8));
    grad_kernel<T><<<unsigned(a.rows * slices), kThreads, (a.top + 3) / 4 * 4 * 12, st>>>(a, slices);
    return cudaGetLastError();
}

tsenor_status finish(cudaError_t e, const char* what) { return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, what); }

constexpr int64_t kMaxRows = int64_t(1) << 24;   // times up to 128 slices: the grid

tsenor_status check_distill(int dtype, const DistillArgs& a) {
    if (dtype != TSENOR_F32 && dtype != TSENOR_BF16) return TSENOR_ERR_ARG;
    if (a.rows < 0 || a.rows > kMaxRows || a.vocab < 1 || a.vocab > TSENOR_DISTILL_MAX_VOCAB ||
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
    cudaStream_t st = (cudaStream_t)stream;
    return finish(dtype == TSENOR_BF16 ? launch_loss<BF16, false>(a, st) : launch_loss<F32, false>(a, st),
                  "tsenor_distill_loss launch");
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
    cudaStream_t st = (cudaStream_t)stream;
    return finish(dtype == TSENOR_BF16 ? launch_loss<BF16, true>(a, st) : launch_loss<F32, true>(a, st),
                  "tsenor_distill_step launch");
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
    cudaStream_t st = (cudaStream_t)stream;
    return finish(dtype == TSENOR_BF16 ? launch_grad<BF16>(a, st) : launch_grad<F32>(a, st),
                  "tsenor_distill_grad launch");
}
