// Distillation from a teacher's top logits, forward and backward.
//
// Row (token) with student logits z, temperature T, teacher entries (i_j, t_j):
//   p_j = exp(t_j / T - c),  c = logsumexp_j(t_j / T) or the teacher's own normaliser
//   q = softmax(z / T),  lse = logsumexp(z / T)
//   loss = T^2 sum_j p_j (log p_j - log q_{i_j})
//   dz_v = w T (P q_v - sum_{j: i_j = v} p_j),  P = sum_j p_j
//
// Bound by memory: z is read from it once and dz written once.  Three kernels:
//   stream_kernel  a row to a CTA, through registers: the loss of many rows, and the step, which reads a row again
//                  (from L2, as a rule), of many rows of up to 192 KB.
//   loss_kernel    a row cut into slices, one to a CTA of a cluster of up to 8: few rows, and the step of longer ones.
//                  Bulk copies bring the slice into shared memory, where its maximum, its sum of exponentials and, for the
//                  step, its gradient are taken, and the CTAs exchange one (maximum, sum, loss term) each.  Slices of up to
//                  64 KB, three CTAs to an SM, overlap one row's loads with another's arithmetic and stores; rows above
//                  512 KB have larger ones, up to 128 KB, and two CTAs or one.  A few rows get more and smaller slices.
//   grad_kernel    the gradient alone, which needs nothing but z and lse (rows of a large lse: a second read).
// Sums over the vocabulary are fp32, the few scalars of a row fp64.  Measured at 2048 x 131072 bf16, 64 entries: loss 95 us
// (5.7 TB/s), step 228 us (4.7 TB/s), gradient 160 us (6.7 TB/s; 240 us where every row has a large lse).
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "pdl.h"
#include "tensor.h"

namespace tsenor {
namespace {

__device__ unsigned long long g_row_failures;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTeachers = 128;                   // further threads of loss_kernel
constexpr int kMaxTop = TSENOR_DISTILL_MAX_TOP;
constexpr int kGroup = 4;                        // chunks of a thread that share a step of the running maximum
constexpr int kSegment = kGroup * kThreads;      // chunks of a slice that are copied under one barrier
constexpr int kMaxSegments = 8;                  // of the largest slice, 128 KB
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
    double inv_t;                                // 1 / temperature
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
        const int all = (vocab - h) / kPer, share = int(unsigned(all + n - 1) / unsigned(n));
        chunk0 = r * share < all ? r * share : all;
        chunks = all - chunk0 < share ? all - chunk0 : share;
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

__device__ __forceinline__ float shuffle_xor(float v, int lane) { return __shfl_xor_sync(kFullMask, v, lane); }

// N threads of a block, from thread FIRST on, that meet at the block's barrier ID.
template <int FIRST, int N, int ID>
struct Team {
    __device__ static int id() { return int(threadIdx.x) - FIRST; }
    __device__ static void sync() { asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory"); }
    __device__ static bool any(bool x) {
        uint32_t r;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\tbar.red.or.pred p, %2, %3, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
                     : "=r"(r) : "r"(uint32_t(x)), "n"(ID), "n"(N) : "memory");
        return r != 0;
    }
    // In a fixed order; the result in every thread.  `red`: N / 32 values that may be used again after the next call.
    template <typename X, typename F>
    __device__ static X reduce(X v, X* red, F f) {
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) v = f(v, shuffle_xor(v, s));
        if ((threadIdx.x & 31) == 0) red[id() / 32] = v;
        sync();
        v = red[0];
#pragma unroll
        for (int k = 1; k < N / 32; ++k) v = f(v, red[k]);
        return v;
    }
};
struct Larger {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Plus {
    template <typename X>
    __device__ X operator()(X a, X b) const { return a + b; }
};

// log of a sum of 1 or more in fp64: the exponent apart, so that logf sees [1, 2). What is not finite is its own log.
__device__ __forceinline__ double log_sum(float s) {
    if (!(s < INFINITY)) return s;
    const int e = int(__float_as_uint(s) >> 23) - 127;
    return double(e) * 0.6931471805599453 + double(logf(__uint_as_float((__float_as_uint(s) & 0x7fffffu) | 0x3f800000u)));
}

// The teacher's entries of a row in shared memory, their number rounded up to 4, and a table to find equal indices,
// which is free again once mark_twins(slice) has run.
template <typename TEAM, int N>
struct Teacher {
    int top, top4, slots;
    float* t;                                    // the teacher's logits (-inf: no entry)
    float* logit;                                // in the same place: the student's logits of the entries' columns
    float* p;
    int* index;                                  // 16-byte aligned; -1: no entry; kTwin set: another entry has it too
    int* table;                                  // of the indices in the slice, open addressing; `slots` a power of two
    static constexpr int kTwin = 1 << 30;        // above every column

    __device__ Teacher(void* at, int* table_, int top_, int slots_)
        : top(top_), top4((top_ + 3) / 4 * 4), slots(slots_), table(table_) {
        t = logit = static_cast<float*>(at);
        p = t + top4;
        index = reinterpret_cast<int*>(p + top4);
    }

    // Reads the entries; empty: none has weight, bad: the row fails.
    __device__ void read_entries(const DistillArgs& a, int64_t row, bool* empty, bool* bad) {
        for (int i = TEAM::id(); i < slots; i += N) table[i] = -1;
        bool wrong = a.teacher_lse && !(fabsf(a.teacher_lse[row]) < INFINITY), any = false;
#pragma unroll 4
        for (int j = TEAM::id(); j < top4; j += N) {
            const int i = j < top ? a.index[row * top + j] : -1;
            const float v = j < top ? a.top_logits[row * top + j] : 0.f;
            const bool in = i >= 0 && i < a.vocab;
            wrong = wrong || (i >= 0 && !(in && v < INFINITY));
            any = any || (in && v > -INFINITY) || i >= a.vocab || (i >= 0 && v != v);
            index[j] = in ? i : -1;
            t[j] = in ? v : -INFINITY;
        }
        *empty = !TEAM::any(any);
        *bad = TEAM::any(wrong) && !*empty;
    }
    // After read_entries: marks the entries in the slice whose index another entry has too.
    template <typename S>
    __device__ void mark_twins(const S& slice) const {
        auto slot = [&](int v, int k) { return table + ((((unsigned(v) * 2654435761u) >> 7) + k) & (slots - 1)); };
        bool met = false;
        for (int j = TEAM::id(); j < top; j += N) {
            const int v = index[j];
            if (v < 0 || !slice.has(v)) continue;
            for (int k = 0; k < slots; ++k) {                                // half of the slots stay free
                const int was = atomicCAS(slot(v, k), -1, v);
                if (was == -1) break;
                if ((was & ~kTwin) == v) {
                    atomicOr(slot(v, k), kTwin);
                    met = true;
                    break;
                }
            }
        }
        if (!TEAM::any(met)) return;             // as a rule
        for (int j = TEAM::id(); j < top; j += N) {
            const int v = index[j];
            if (v < 0 || !slice.has(v)) continue;
            for (int k = 0; k < slots; ++k) {
                const int was = *slot(v, k);
                if ((was & ~kTwin) != v) continue;
                index[j] = was;
                break;
            }
        }
    }
    // After read_entries: p of this thread's entries; P = sum p, and c of log p_j = t_j / T - c.  `red`: 2 N / 32 values.
    __device__ float weights(const DistillArgs& a, int64_t row, float* red, double* c) const {
        float total = 1.f;                       // of a softmax over the entries
        if (a.teacher_lse) {
            *c = double(a.teacher_lse[row]);
        } else {
            const float inv_t = 1.f / a.temperature;
            float high = -INFINITY, sum = 0.f;
            for (int j = TEAM::id(); j < top; j += N) high = fmaxf(high, t[j]);
            high = TEAM::reduce(high, red, Larger());
            for (int j = TEAM::id(); j < top; j += N) sum += expf((t[j] - high) * inv_t);
            *c = double(high) * a.inv_t + log_sum(TEAM::reduce(sum, red + N / 32, Plus()));
        }
        float part = 0.f;
        for (int j = TEAM::id(); j < top4; j += N) {
            const float w = t[j] == -INFINITY ? 0.f : expf(float(double(t[j]) * a.inv_t - *c));
            p[j] = w;
            part += w;
        }
        if (a.teacher_lse) total = TEAM::reduce(part, red, Plus());
        return total;
    }
    // Thread `me` of M: f(j, v, sum of the weights of index v) for the entries in a slice, each index once.
    template <int M, typename S, typename F>
    __device__ __forceinline__ void each(int me, const S& slice, F f) const {
        for (int j = me; j < top; j += M) {
            const int i = index[j], v = i & ~kTwin;
            if (i < 0 || !slice.has(v)) continue;
            bool first = true;
            float w = p[j];
            if (i & kTwin) {                     // in the order of the entries
                w = 0.f;
                for (int k = 0; k < top4; k += 4) {
                    const int4 o = *reinterpret_cast<const int4*>(index + k);
                    if (o.x == i) { first = first && k >= j; w += p[k]; }
                    if (o.y == i) { first = first && k + 1 >= j; w += p[k + 1]; }
                    if (o.z == i) { first = first && k + 2 >= j; w += p[k + 2]; }
                    if (o.w == i) { first = first && k + 3 >= j; w += p[k + 3]; }
                }
            }
            if (first) f(j, v, w);
        }
    }
};

constexpr int slots_of(int top) {
    int n = 32;
    while (n < 2 * top) n *= 2;
    return n;
}
// Shared memory of `rows` rows' entries and a table.
constexpr unsigned teacher_bytes(int top, int rows) { return unsigned(rows * ((top + 3) / 4 * 4) * 12 + slots_of(top) * 4); }

// Gradient 0 for the columns of a slice.
template <typename T, int M>
__device__ void write_zeros(typename T::storage* g, const Slice<T>& slice, bool vec) {
    if (vec) {
        uint4* o = reinterpret_cast<uint4*>(g + slice.first);
        for (int i = threadIdx.x; i < slice.chunks; i += M) o[i] = make_uint4(0, 0, 0, 0);
    } else {
        for (int i = threadIdx.x; i < slice.chunks * Slice<T>::kPer; i += M) write<T>(g + slice.first + i, 0.f);
    }
    for (int i = threadIdx.x; i < slice.extras(); i += M) write<T>(g + slice.extra(i), 0.f);
}

// One chunk of gradient from f(logit) of its entries.  LAST: it should not push from L2 what will be read again.
template <typename T, bool LAST = false, typename F>
__device__ __forceinline__ void write_chunk(typename T::storage* g, const uint4& z, bool vec, F f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < Slice<T>::kPer / 2; ++i) set_pair<T>(w, i, f(pair_of<T>(z, i)));
    if (vec) {
        if (LAST) __stcs(reinterpret_cast<uint4*>(g), make_uint4(w[0], w[1], w[2], w[3]));
        else *reinterpret_cast<uint4*>(g) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < Slice<T>::kPer; ++k) {
            if constexpr (std::is_same<T, BF16>::value) g[k] = uint16_t(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
            else g[k] = __uint_as_float(w[k]);
        }
    }
}

// A softmax normaliser in units of z: sum of 2^((z - high) scale), where `high` counts as the nearest finite
// value.  A part without a finite logit has high -inf and sum 0; a +inf makes the sum +inf, a NaN anywhere makes
// it NaN.  All of it survives the joins.
struct Norm {
    float high, sum;
};
__device__ __forceinline__ float finite_base(float high) { return fminf(fmaxf(high, -FLT_MAX), FLT_MAX); }
// `n` normalisers, read through get(k).
template <typename F>
__device__ __forceinline__ Norm join(int n, float scale2, F get) {
    Norm all{-INFINITY, 0.f};
    for (int k = 0; k < n; ++k) all.high = fmaxf(all.high, get(k).high);
    const float base = finite_base(all.high);
    for (int k = 0; k < n; ++k) {
        const Norm o = get(k);
        all.sum += o.sum * ex2((o.high - base) * scale2);
    }
    return all;
}
// Adds n chunks to a normaliser: their maximum first, so that one step of the running maximum serves them all.
template <typename T, int n>
__device__ __forceinline__ void take(Norm& norm, const uint4* v, float scale2) {
    float high;
    if constexpr (std::is_same<T, BF16>::value) {
        uint32_t m = v[0].x;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            uint32_t x, y;
            asm("max.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(v[k].x), "r"(v[k].y));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(v[k].z), "r"(v[k].w));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(y));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x));
        }
        high = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        high = __uint_as_float(v[0].x);
#pragma unroll
        for (int k = 0; k < n; ++k)
            high = fmaxf(fmaxf(high, fmaxf(__uint_as_float(v[k].x), __uint_as_float(v[k].y))),
                         fmaxf(__uint_as_float(v[k].z), __uint_as_float(v[k].w)));
    }
    high = fmaxf(norm.high, high);
    const float base = finite_base(high);
    const float2 minus = make_float2(-base, -base), by2 = make_float2(scale2, scale2);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int k = 0; k < n; ++k)
#pragma unroll
        for (int q = 0; q < Slice<T>::kPer / 2; ++q) {
            const float2 x = mul2(add2(pair_of<T>(v[k], q), minus), by2);
            sum[q & 1] = add2(sum[q & 1], make_float2(ex2(x.x), ex2(x.y)));
        }
    const float2 both = add2(sum[0], sum[1]);
    norm.sum = fmaf(norm.sum, ex2((norm.high - base) * scale2), both.x + both.y);
    norm.high = high;
}
// Adds one entry.
__device__ __forceinline__ void take_one(Norm& norm, float x, float scale2) {
    const Norm two[2] = {norm, Norm{x == x ? x : -INFINITY, x == x ? (x == -INFINITY ? 0.f : 1.f) : x}};
    norm = join(2, scale2, [&](int k) { return two[k]; });
}
// Over a warp, in every lane.
__device__ __forceinline__ Norm warp_join(Norm norm, float scale2) {
    float high = norm.high;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) high = fmaxf(high, __shfl_xor_sync(kFullMask, high, s));
    norm.sum *= ex2((norm.high - finite_base(high)) * scale2);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) norm.sum += __shfl_xor_sync(kFullMask, norm.sum, s);
    return Norm{high, norm.sum};
}

// A row's loss is T^2 (sum_j p_j (log p_j - z_j / T) + lse sum_j p_j): both sums, over a slice's entries, in fp64, since they
// all but cancel where the student is near its teacher.
struct Terms {
    double gap, mass;
    __device__ Terms operator+(Terms o) const { return Terms{gap + o.gap, mass + o.mass}; }
};
__device__ __forceinline__ Terms shuffle_xor(Terms s, int lane) {
    return Terms{__shfl_xor_sync(kFullMask, s.gap, lane), __shfl_xor_sync(kFullMask, s.mass, lane)};
}
// By the threads of a team, which also keep the entries' logits.  `red`: N / 32 values.
template <typename T, typename TEAM, int N>
__device__ Terms team_terms(const DistillArgs& a, const typename T::storage* z, const Slice<T>& slice,
                            const Teacher<TEAM, N>& teacher, double c, Terms* red) {
    Terms s{0.0, 0.0};
#pragma unroll 4
    for (int j = TEAM::id(); j < a.top; j += N) {
        const int i = teacher.index[j], v = i & ~Teacher<TEAM, N>::kTwin;
        const float w = teacher.p[j];
        if (i < 0 || !slice.has(v)) continue;
        const float x = read<T>(z + v);
        if (w > 0.f) {
            s.gap += double(w) * ((double(teacher.t[j]) - double(x)) * a.inv_t - c);
            s.mass += double(w);
        }
        teacher.logit[j] = x;
    }
    return TEAM::reduce(s, red, Plus());
}

// What a slice tells the others of its row.
struct alignas(16) Share {
    Terms terms;
    Norm norm;
};

// One thread: the row's loss (and lse), its failure.
template <bool STEP>
__device__ void write_loss(const DistillArgs& a, int64_t row, Norm norm, Terms s, bool empty, bool failed) {
    const double lse = norm.high == -INFINITY ? double(norm.high + norm.sum)      // no finite logit: -inf, or NaN
                                              : double(norm.high) * a.inv_t + log_sum(norm.sum);
    a.loss[row] = failed ? NAN : empty ? 0.f
                  : float(double(a.temperature) * double(a.temperature) * (s.gap + s.mass * lse));
    if (!STEP) a.lse[row] = failed ? NAN : float(lse);
    if (failed) atomicAdd(&g_row_failures, 1ull);
}

// Loss (STEP: and gradient).  A cluster of `slices` CTAs walks the rows, one slice to a CTA.
// Eight warps work on the slice in shared memory.  Four more are a row ahead: they see to the teacher's entries
// and start the copy of each segment as soon as the workers have written the gradient of the one that it
// replaces, so that reading, arithmetic and writing overlap within a CTA too.
//   full[s]   segment s of this row is there          free[s]  its workers are done with it
//   told[b]   the entries of a row (two buffers)      done[b]  its workers are done with them
//   joined[j] the shares of all slices of the row
// 2048 x 131072 bf16 228 us (4.7 TB/s), 1024 x 131072 fp32 202 us (5.3 TB/s; 10 % more with a CTA for each slice of each row).
template <typename T, bool STEP>
__global__ void __launch_bounds__(kThreads + kTeachers, 3)
loss_kernel(const DistillArgs a, const int slices, const int chunk_room, const int slots) {
    extern __shared__ __align__(128) uint4 chunk[];
    constexpr int kPer = Slice<T>::kPer;
    __shared__ Share share[2][kMaxSlices];
    __shared__ Norm part[2][kWarps];
    __shared__ Terms red64[kTeachers / 32], terms_of_slice[2];
    __shared__ float red[2 * kTeachers / 32], total_of_p[2], extra[2][2 * kPer];
    __shared__ int flags[2];                     // 1: no entry, 2: the row fails
    __shared__ float row_high[2], row_scale[2], row_by[2];                    // of a row's gradient; by 0: it is 0
    __shared__ uint64_t full[kMaxSegments], free[kMaxSegments], told[2], done[2], joined[2];
    using Extra = Team<kThreads, kTeachers, 1>;
    using Workers = Team<0, kThreads, 2>;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = slices > 1 ? int(cluster_rank()) : 0;
    const int64_t first = blockIdx.x / unsigned(slices), step = gridDim.x / unsigned(slices);
    const int segments = (chunk_room + kSegment - 1) / kSegment;
    const float inv_t = 1.f / a.temperature, scale2 = inv_t * kLog2E;
    if (t == 0) {
        for (int i = 0; i < segments; ++i) {
            mbar_init(full + i, 1);
            mbar_init(free + i, kWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(told + b, kTeachers / 32);
            mbar_init(done + b, kWarps);
            mbar_init(joined + b, slices);
        }
        mbar_init_fence();
    }
    let_next_start();
    if (slices > 1) cluster_sync();              // peers write here
    else __syncthreads();
    prior_done();
    auto row_of = [&](int64_t row) { return static_cast<const typename T::storage*>(a.logits) + row * a.ld; };
    auto teacher_of = [&](int b) {
        float* at = reinterpret_cast<float*>(chunk + chunk_room);
        const int words = (a.top + 3) / 4 * 4 * 3;
        return Teacher<Extra, kTeachers>(at + b * words, reinterpret_cast<int*>(at + 2 * words), a.top, slots);
    };
    bool stalled = false;

    if (warp >= kWarps) {
        unsigned i = 0, newest = 0;              // the row (its number here) of the newest copies,
        int copied = 0;                          // and how many of its segments they bring; in the warp that copies
        // the columns of a row's entries, once the workers have written the row (its number here: n)
        auto write_targets = [&](int64_t row, unsigned n) {
            const int b = n & 1;
            if (!warp_sleep(done + b, (n >> 1) & 1)) return false;
            if (!STEP || row_by[b] == 0.f) return true;
            const float scale = row_scale[b], m = row_high[b], by = row_by[b];
            auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
            const Slice<T> slice(row_of(row), int(a.vocab), rank, slices);
            const Teacher<Extra, kTeachers> teacher = teacher_of(b);
            teacher.template each<kTeachers>(Extra::id(), slice, [&](int j, int v, float w) {
                write<T>(g + v, scale * ex2((teacher.logit[j] - m) * scale2) - by * w);
            });
            return true;
        };
        for (int64_t row = first; row < a.rows; row += step, ++i) {
            const int b = i & 1;
            const auto* z = row_of(row);
            const Slice<T> slice(z, int(a.vocab), rank, slices);
            Teacher<Extra, kTeachers> teacher = teacher_of(b);
            bool empty, bad;
            teacher.read_entries(a, row, &empty, &bad);
            if (t == kThreads) flags[b] = (empty ? 1 : 0) | (bad ? 2 : 0);
            const bool skip = STEP && (empty || bad);                         // the logits are not read
            // segments past the slice complete at once, as all do without bytes
            auto copy = [&](int s) {
                const int c = s * kSegment, left = slice.chunks - c;
                const int n = skip || left < 0 ? 0 : left < kSegment ? left : kSegment;
                mbar_arrive_expect_tx(full + s, n * 16);
                if (n > 0) bulk_load(chunk + c, z + slice.first + c * kPer, n * 16, full + s);
            };
            if (i == 0 && t == kThreads)
                for (int s = 0; s < segments; ++s) copy(s);
            if (i == 0) copied = segments;
            const int e = t - kThreads;
            if (e < slice.extras()) extra[b][e] = read<T>(z + slice.extra(e));
            if (!empty && !(STEP && bad)) {
                if (STEP) teacher.mark_twins(slice);
                double c;
                const float total = teacher.weights(a, row, red, &c);
                const Terms terms = team_terms<T>(a, z, slice, teacher, c, red64);
                if (t == kThreads) {
                    total_of_p[b] = total;
                    terms_of_slice[b] = terms;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(told + b);
            if (i > 0 && warp == kWarps) {
                newest = i;
                for (copied = 0; copied < segments; ++copied) {
                    if (!warp_sleep(free + copied, (i - 1) & 1)) { stalled = true; break; }
                    if (lane == 0) copy(copied);
                    __syncwarp();
                }
            }
            if (i > 0 && !write_targets(row - step, i - 1)) stalled = true;
            if (Extra::any(stalled)) { stalled = true; break; }
        }
        if (STEP && i > 0 && !stalled && !write_targets(first + (i - 1) * step, i - 1)) stalled = true;
        // copies in flight end before the block does, whichever warp gave up
        if (warp == kWarps)
            for (int s = 0; s < segments; ++s)
                if ((s < copied || newest > 0) && !warp_drain(full + s, (s < copied ? newest : newest - 1) & 1)) stalled = true;
    } else {
        unsigned i = 0, joins = 0;
        for (int64_t row = first; row < a.rows; row += step, ++i) {
            const int b = i & 1;
            const auto* z = row_of(row);
            auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
            const Slice<T> slice(z, int(a.vocab), rank, slices);
            const bool vec = STEP && ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
            auto leave = [&](uint64_t* bar) {    // this warp is done with what the barrier stands for
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            // one pass over the slice; a NaN or +inf anywhere makes the sum one too
            Norm norm{-INFINITY, 0.f};
            for (int s = 0; s < segments; ++s) {
                if (!warp_sleep(full + s, i & 1)) { stalled = true; break; }
                // Written before the first segment began.  A row that is not read waits for its (empty) segments all the
                // same: its arrivals on free[s] must not overtake the copying warp's wait on them.
                if (STEP && flags[b]) continue;
                const uint4* from = chunk + s * kSegment + t;
                const int left = slice.chunks - s * kSegment - t;
                if (left > (kGroup - 1) * kThreads) {
                    uint4 v[kGroup];
#pragma unroll
                    for (int k = 0; k < kGroup; ++k) v[k] = from[k * kThreads];
                    take<T, kGroup>(norm, v, scale2);
                } else {
                    for (int k = 0; k * kThreads < left; ++k) {
                        const uint4 v = from[k * kThreads];
                        take<T, 1>(norm, &v, scale2);
                    }
                }
                if (!STEP) leave(free + s);
            }
            if (!warp_sleep(told + b, (i >> 1) & 1)) stalled = true;
            if (Workers::any(stalled)) { stalled = true; break; }
            const bool empty = flags[b] & 1;
            bool failed = flags[b] & 2;
            if (STEP && flags[b]) {
                for (int s = 0; s < segments; ++s) leave(free + s);
                write_zeros<T, kThreads>(g, slice, vec);
                if (t == 0 && rank == 0) {
                    a.loss[row] = failed ? NAN : 0.f;
                    if (failed) atomicAdd(&g_row_failures, 1ull);
                }
                if (t == 0) row_by[b] = 0.f;
                leave(done + b);
                continue;
            }
            if (t < slice.extras()) take_one(norm, extra[b][t], scale2);
            norm = warp_join(norm, scale2);
            if (lane == 0) part[b][warp] = norm;
            Workers::sync();
            norm = join(kWarps, scale2, [&](int k) { return part[b][k]; });
            Terms terms = empty ? Terms{0.0, 0.0} : terms_of_slice[b];
            const float total = empty ? 0.f : total_of_p[b];
            if (slices > 1) {
                const int j = joins & 1;
                if (t < slices) {
                    const uint32_t to = cluster_addr(smem_u32(&share[j][rank]), t);
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to + 16), "f"(norm.high), "f"(norm.sum) : "memory");
                    asm volatile("st.shared::cluster.v2.f64 [%0], {%1, %2};" ::"r"(to), "d"(terms.gap), "d"(terms.mass) : "memory");
                    cluster_arrive(cluster_addr(smem_u32(joined + j), t));
                }
                if (!warp_cluster_sleep(joined + j, (joins >> 1) & 1)) stalled = true;
                if (Workers::any(stalled)) { stalled = true; break; }
                ++joins;
                norm = join(slices, scale2, [&](int k) { return share[j][k].norm; });
                terms = Terms{0.0, 0.0};
                for (int k = 0; k < slices; ++k) {
                    terms.gap += share[j][k].terms.gap;
                    terms.mass += share[j][k].terms.mass;
                }
            }
            const float m = norm.high;
            failed = failed || (!empty && !(fabsf(m) < INFINITY && norm.sum < INFINITY));
            if (t == 0 && rank == 0) write_loss<STEP>(a, row, norm, terms, empty, failed);
            if constexpr (STEP) {
                const float by = a.temperature * (a.weight ? a.weight[row] : 1.f);
                if (failed || by == 0.f) {
                    for (int s = 0; s < segments; ++s) leave(free + s);
                    write_zeros<T, kThreads>(g, slice, vec);
                } else {
                    const float scale = by * total / norm.sum;
                    const float2 minus_m = make_float2(-m, -m), scale_2 = make_float2(scale, scale),
                                 by2 = make_float2(scale2, scale2);
                    for (int s = 0; s < segments; ++s) {
                        auto gradient = [&](float2 x) {
                            x = mul2(add2(x, minus_m), by2);
                            return mul2(make_float2(ex2(x.x), ex2(x.y)), scale_2);
                        };
                        const uint4* from = chunk + s * kSegment + t;
                        auto* to = g + slice.first + (s * kSegment + t) * kPer;
                        const int left = slice.chunks - s * kSegment - t;
                        if (left > (kGroup - 1) * kThreads) {
                            uint4 v[kGroup];
#pragma unroll
                            for (int k = 0; k < kGroup; ++k) v[k] = from[k * kThreads];
#pragma unroll
                            for (int k = 0; k < kGroup; ++k) write_chunk<T>(to + k * kThreads * kPer, v[k], vec, gradient);
                        } else {
                            for (int k = 0; k * kThreads < left; ++k)
                                write_chunk<T>(to + k * kThreads * kPer, from[k * kThreads], vec, gradient);
                        }
                        leave(free + s);
                    }
                    if (t < slice.extras()) write<T>(g + slice.extra(t), scale * ex2((extra[b][t] - m) * scale2));
                }
                if (t == 0) {
                    row_high[b] = m;
                    row_scale[b] = by * total / norm.sum;
                    row_by[b] = failed ? 0.f : by;
                }
            }
            leave(done + b);
        }
    }
    if (stalled && lane == 0) atomicAdd(&g_row_failures, 1ull);
    __syncwarp();
    if (slices > 1) cluster_sync();              // no peer writes here any more
}

// The same with one CTA to a row, which streams it through registers, twice for the step
// (the second time from L2, last chunks first).  W threads take the row, E its entries.  Nothing of a row waits for
// another SM, and a row's fixed costs are paid once.
template <typename T, bool STEP, int W, int E>
__global__ void __launch_bounds__(W + E, (STEP ? 1920 : 1536) / (W + E))
stream_kernel(const DistillArgs a, const int slots) {
    extern __shared__ __align__(128) uint4 room[];
    __shared__ Norm part[W / 32];
    __shared__ Terms red64[E / 32], terms_of_row;
    __shared__ float total_of_p, red[2 * E / 32];
    __shared__ int flags;                        // 1: no entry, 2: the row fails
    constexpr int kPer = Slice<T>::kPer;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t row = blockIdx.x;
    const auto* z = static_cast<const typename T::storage*>(a.logits) + row * a.ld;
    auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
    const Slice<T> slice(z, int(a.vocab), 0, 1);
    using Extra = Team<W, E, 1>;
    Teacher<Extra, E> teacher(room, reinterpret_cast<int*>(room) + (a.top + 3) / 4 * 4 * 3, a.top, slots);
    const bool vec = STEP && ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    const float inv_t = 1.f / a.temperature, scale2 = inv_t * kLog2E;
    const uint4* in = reinterpret_cast<const uint4*>(z + slice.first);
    let_next_start();
    prior_done();
    if (warp >= W / 32) {
        bool empty, bad;
        teacher.read_entries(a, row, &empty, &bad);
        if (t == W) flags = (empty ? 1 : 0) | (bad ? 2 : 0);
        if (STEP) __syncthreads();
        if (!empty && !(STEP && bad)) {
            if (STEP) teacher.mark_twins(slice);
            double c;
            const float total = teacher.weights(a, row, red, &c);
            const Terms terms = team_terms<T>(a, z, slice, teacher, c, red64);
            if (t == W) {
                total_of_p = total;
                terms_of_row = terms;
            }
        }
    } else {
        if (STEP) __syncthreads();
        if (!(STEP && flags)) {
            // a NaN or +inf anywhere makes the sum one too
            Norm norm{-INFINITY, 0.f};
            int c = t;
            for (; c + (kGroup - 1) * W < slice.chunks; c += kGroup * W) {
                uint4 v[kGroup];
#pragma unroll
                for (int k = 0; k < kGroup; ++k) v[k] = in[c + k * W];
                take<T, kGroup>(norm, v, scale2);
            }
            for (; c < slice.chunks; c += W) {
                const uint4 v = in[c];
                take<T, 1>(norm, &v, scale2);
            }
            if (t < slice.extras()) take_one(norm, read<T>(z + slice.extra(t)), scale2);
            norm = warp_join(norm, scale2);
            if (lane == 0) part[warp] = norm;
        }
    }
    __syncthreads();
    const bool empty = flags & 1;
    bool failed = flags & 2;
    if (STEP && flags) {
        if (warp < W / 32) write_zeros<T, W>(g, slice, vec);
        if (t == 0) {
            a.loss[row] = failed ? NAN : 0.f;
            if (failed) atomicAdd(&g_row_failures, 1ull);
        }
        return;
    }
    const Norm norm = join(W / 32, scale2, [&](int k) { return part[k]; });
    const float m = norm.high;
    failed = failed || (!empty && !(fabsf(m) < INFINITY && norm.sum < INFINITY));
    if (t == W) write_loss<STEP>(a, row, norm, empty ? Terms{0.0, 0.0} : terms_of_row, empty, failed);
    if constexpr (STEP) {
        const float by = a.temperature * (a.weight ? a.weight[row] : 1.f);
        if (failed || by == 0.f) {
            if (warp < W / 32) write_zeros<T, W>(g, slice, vec);
            return;
        }
        const float scale = by * total_of_p / norm.sum;
        auto at = [&](float x) { return scale * ex2((x - m) * scale2); };
        const float2 minus_m = make_float2(-m, -m), scale_2 = make_float2(scale, scale), by2 = make_float2(scale2, scale2);
        auto both = [&](float2 x) {
            x = mul2(add2(x, minus_m), by2);
            return mul2(make_float2(ex2(x.x), ex2(x.y)), scale_2);
        };
        if (warp < W / 32) {
            int c = slice.chunks - 1 - t;
            for (; c - (kGroup - 1) * W >= 0; c -= kGroup * W) {
                uint4 v[kGroup];
#pragma unroll
                for (int k = 0; k < kGroup; ++k) v[k] = __ldcs(in + c - k * W);
#pragma unroll
                for (int k = 0; k < kGroup; ++k)
                    write_chunk<T, true>(g + slice.first + (c - k * W) * kPer, v[k], vec, both);
            }
            for (; c >= 0; c -= W) write_chunk<T, true>(g + slice.first + c * kPer, __ldcs(in + c), vec, both);
            if (t < slice.extras()) write<T>(g + slice.extra(t), at(read<T>(z + slice.extra(t))));
        }
        __syncthreads();                         // the entries' columns are written again
        if (warp < W / 32)
            teacher.template each<W>(t, slice, [&](int j, int v, float w) { write<T>(g + v, at(teacher.logit[j]) - by * w); });
    }
}

// A whole row's normaliser by the threads of a block, in every thread.
template <typename T>
__device__ Norm block_norm(const typename T::storage* z, const Slice<T>& row, float scale2, Norm* part) {
    const uint4* in = reinterpret_cast<const uint4*>(z + row.first);
    Norm norm{-INFINITY, 0.f};
    int c = threadIdx.x;
    for (; c + (kGroup - 1) * kThreads < row.chunks; c += kGroup * kThreads) {
        uint4 v[kGroup];
#pragma unroll
        for (int k = 0; k < kGroup; ++k) v[k] = in[c + k * kThreads];
        take<T, kGroup>(norm, v, scale2);
    }
    for (; c < row.chunks; c += kThreads) {
        const uint4 v = in[c];
        take<T, 1>(norm, &v, scale2);
    }
    if (threadIdx.x < row.extras()) take_one(norm, read<T>(z + row.extra(threadIdx.x)), scale2);
    norm = warp_join(norm, scale2);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = norm;
    __syncthreads();
    return join(kWarps, scale2, [&](int k) { return part[k]; });
}

// The gradient from lse; blockIdx.x is a row's slice.
// q = exp(z / T - lse) as unit * 2^((z - base) log2(e) / T): base = T lse in fp32, what its rounding leaves in `unit`, so that the
// error of q is that of lse itself, 2^-24 |lse|, and some 2^-22.  A larger lse (low temperatures, logits far from 0) or a T lse past
// fp32 is not used: the row's first block takes the row by itself, maximum and sum anew from one more read, as the step has them.
constexpr float kNearLse = 64.f;
template <typename T>
__global__ void __launch_bounds__(kThreads) grad_kernel(const DistillArgs a, const int slices, const int slots) {
    extern __shared__ __align__(128) uint4 room[];
    __shared__ float red[2 * kWarps];
    __shared__ Norm part[kWarps];
    constexpr int kPer = Slice<T>::kPer;
    constexpr int kAhead = 4;                    // chunks of a thread in flight
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x / slices;
    const int rank = int(blockIdx.x % slices);
    const auto* z = static_cast<const typename T::storage*>(a.logits) + row * a.ld;
    auto* g = static_cast<typename T::storage*>(a.grad) + row * a.ldg;
    Slice<T> slice(z, int(a.vocab), rank, slices);
    Teacher<Team<0, kThreads, 1>, kThreads> teacher(room, reinterpret_cast<int*>(room) + (a.top + 3) / 4 * 4 * 3, a.top, slots);
    float* target = teacher.logit;               // the gradients of the entries' columns
    const bool vec = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    let_next_start();
    prior_done();
    const float lse = a.lse[row], scale2 = 1.f / a.temperature * kLog2E;
    const double middle = double(lse) * double(a.temperature);
    const float by = a.temperature * (a.weight ? a.weight[row] : 1.f);
    float base = float(middle), unit = expf(float((double(base) - middle) * a.inv_t));
    bool empty, bad;
    teacher.read_entries(a, row, &empty, &bad);
    bad = bad || (!empty && lse != lse);
    if (!bad && !empty && !(fabsf(lse) <= kNearLse && fabsf(base) <= FLT_MAX)) {
        if (rank > 0) return;
        slice = Slice<T>(z, int(a.vocab), 0, 1);
        const Norm norm = block_norm<T>(z, slice, scale2, part);
        bad = !(fabsf(norm.high) < INFINITY && norm.sum < INFINITY);
        base = norm.high;
        unit = 1.f / norm.sum;
    }
    if (bad && rank == 0 && t == 0) atomicAdd(&g_row_failures, 1ull);
    if (bad || empty || by == 0.f) {
        write_zeros<T, kThreads>(g, slice, vec);
        return;
    }
    const uint4* in = reinterpret_cast<const uint4*>(z + slice.first);
    uint4 v[kAhead];
    auto load = [&](int c) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c + i * kThreads < slice.chunks) v[i] = in[c + i * kThreads];
    };
    load(t);                                     // on their way while the weights are made
    teacher.mark_twins(slice);
    double c;
    const float total = teacher.weights(a, row, red, &c);
    __syncthreads();
    const float scale = by * total * unit;
    auto at = [&](float x) { return scale * ex2((x - base) * scale2); };
    // the entries' gradients before anything is written: grad may be the logits
    teacher.template each<kThreads>(t, slice, [&](int j, int c, float w) { target[j] = at(read<T>(z + c)) - by * w; });
    __syncthreads();
    const float2 minus = make_float2(-base, -base), by2 = make_float2(scale2, scale2), scale_2 = make_float2(scale, scale);
    for (int c = t; c < slice.chunks; c += kAhead * kThreads) {
        if (c != t) load(c);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c + i * kThreads < slice.chunks)
                write_chunk<T>(g + slice.first + (c + i * kThreads) * kPer, v[i], vec, [&](float2 x) {
                    x = mul2(add2(x, minus), by2);
                    return mul2(make_float2(ex2(x.x), ex2(x.y)), scale_2);
                });
    }
    if (t < slice.extras()) write<T>(g + slice.extra(t), at(read<T>(z + slice.extra(t))));
    __syncthreads();
    teacher.template each<kThreads>(t, slice, [&](int j, int c, float) { write<T>(g + c, target[j]); });
}

// Slices of a row: at most kSliceBytes each (larger in rows that kMaxSlices of those do not hold), and for few rows enough CTAs to fill the
// device twice, of 4 KB at least.
int slices_of(int64_t rows, int64_t row_bytes) {
    int n = 1;
    while (n < kMaxSlices && (row_bytes > int64_t(n) * kSliceBytes || (rows * n < 296 && row_bytes > int64_t(n) * 8192))) n *= 2;
    return n;
}

// Streaming pays where a row's fixed costs weigh more than a second read: for the loss
// (which has none) wherever the rows fill the device, 93 us against 139 for 2048 x 131072 bf16; for the step as long as
// the rows in work stay in L2, five to an SM, which second reads and stores marked as the last use help: 18 us
// against 57 for 4096 x 1000 bf16, 58 against 62 for 2048 x 32000, 148 against 182 for 2048 x 80000, 142 against 155
// for 2048 x 40000 fp32, but 182 against 175 for 2048 x 50000 fp32 and 243 against 236 for 2048 x 131072 bf16.
constexpr int64_t kStepRow = 192 * 1024;
bool streams(bool step, int64_t rows, int64_t row_bytes) { return rows >= 148 && (!step || row_bytes <= kStepRow); }

// Threads of a streaming CTA: on the row, and on its entries.  Short rows wait for the entries, so that where
// there are more rows than the wide CTAs that run at once, smaller ones, more to an SM, pay: with 64 entries 18 us
// for a step of 4096 x 1000 bf16 against 33, 13 against 24 for its loss, 19 against 29 for the loss of 4096 x 8000.
// Long rows want the loads of a wide CTA (the loss of 2048 x 131072 takes 93 us and would take 108), many entries
// its threads (1000 of them, 512 x 2000: 21 and would take 29).
constexpr int64_t kShortRow = 32 * 1024;
constexpr int kNarrow = 96, kNarrowTeachers = 64;

template <typename T, bool STEP, int W, int E>
cudaError_t launch_stream(const DistillArgs& a, cudaStream_t st) {
    return launch_early(stream_kernel<T, STEP, W, E>, a.rows, W + E, teacher_bytes(a.top, 1), 1, st, a, slots_of(a.top));
}

template <typename T, bool STEP>
cudaError_t launch_loss(const DistillArgs& a, cudaStream_t st) {
    const int64_t row_bytes = a.vocab * int64_t(sizeof(typename T::storage));
    if (streams(STEP, a.rows, row_bytes)) {
        return row_bytes <= kShortRow && a.rows > 4 * 148 ? launch_stream<T, STEP, kNarrow, kNarrowTeachers>(a, st)
                                                          : launch_stream<T, STEP, kThreads, kTeachers>(a, st);
    }
    const int slices = slices_of(a.rows, row_bytes);
    const int chunk_room = int((row_bytes / 16 + slices - 1) / slices);
    const unsigned bytes = unsigned(chunk_room * 16) + teacher_bytes(a.top, 2);
    constexpr unsigned most = kMaxSegments * kSegment * 16 + teacher_bytes(kMaxTop, 2);
    static_assert(most + 4096 <= 227 * 1024, "shared memory of a CTA");
    cudaError_t e = allow_shared(loss_kernel<T, STEP>, most);
    if (e != cudaSuccess) return e;
    // No more clusters than run at once, or the last ones would start when the others are through.
    int64_t clusters = a.rows;
    if (clusters * slices > 148) {
        int fit = 0;
        e = clusters_that_fit(&fit, loss_kernel<T, STEP>, kThreads + kTeachers, bytes, slices);
        if (e != cudaSuccess) return e;
        if (fit > 0 && clusters > fit) clusters = fit;
    }
    return launch_early(loss_kernel<T, STEP>, clusters * slices, kThreads + kTeachers, bytes, slices, st, a, slices, chunk_room,
                        slots_of(a.top));
}

template <typename T>
cudaError_t launch_grad(const DistillArgs& a, cudaStream_t st) {
    // about 64 KB to a CTA: the teacher's weights are computed for each
    const int64_t row_bytes = a.vocab * int64_t(sizeof(typename T::storage));
    const int slices = a.rows >= 296 ? int((row_bytes + kSliceBytes - 1) / kSliceBytes)
                                     : int((row_bytes + kSliceBytes / 8 - 1) / (kSliceBytes / 8));
    return launch_early(grad_kernel<T>, a.rows * slices, kThreads, teacher_bytes(a.top, 1), 1, st, a, slices, slots_of(a.top));
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

#ifdef TSENOR_GIVE_UP
extern "C" int give_up_distillation(unsigned polls, unsigned one_in) { return give_up(polls, one_in); }
#endif

cudaError_t row_failures(unsigned long long** counter) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(counter), g_row_failures);
}

}  // namespace tsenor

using namespace tsenor;

extern "C" tsenor_status tsenor_distill_loss(const void* logits, tsenor_dtype dtype, int64_t rows, int64_t vocab,
                                             int64_t ld, const int32_t* index, const float* top_logits, int top,
                                             const float* teacher_lse, float temperature, float* loss, float* lse,
                                             tsenor_stream_t stream) {
    const DistillArgs a{logits, rows, vocab, ld, index, top_logits, top, teacher_lse, temperature, 1.0 / temperature,
                        nullptr, loss, lse,
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
    const DistillArgs a{logits, rows, vocab, ld, index, top_logits, top, teacher_lse, temperature, 1.0 / temperature,
                        weight, loss, nullptr, grad, ldg};
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
    const DistillArgs a{logits, rows, vocab, ld, index, top_logits, top, teacher_lse, temperature, 1.0 / temperature,
                        weight, nullptr, const_cast<float*>(lse), grad, ldg};
    const tsenor_status s = check_distill(dtype, a);
    if (s != TSENOR_OK || rows == 0) return s;
    if (!lse || !aligned(lse, 4) || !grad_ok(dtype, a)) return TSENOR_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    return finish(dtype == TSENOR_BF16 ? launch_grad<BF16>(a, st) : launch_grad<F32>(a, st),
                  "tsenor_distill_grad launch");
}
