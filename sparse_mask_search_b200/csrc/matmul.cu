// Product of two e4m3 matrices with a power-of-two scale per block of 128 along
// the contracted axis:
//   nt  out[m,n] = sum_k A[m,k] B[n,k]     nn  A[m,k] B[k,n]     tn  A[k,m] B[k,n]
#include "common.cuh"
#include "host.h"

namespace tsenor {
namespace {

struct MatmulArgs {
    const uint8_t *a, *b;
    int64_t lda, ldb;
    const uint8_t *sa, *sb;
    int64_t m, n, k;
    const uint32_t* mask;
    int64_t wpr;
    void* out;
    int64_t ldo;
    bool a_t, b_t;          // the operand is stored with its contracted axis along rows
    bool bf16;
};

__device__ __forceinline__ float decode(uint32_t u) {
    const uint32_t e = (u >> 3) & 15u, f = u & 7u;
    float x = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : float(f) * 0.001953125f;
    if ((u & 127u) == 127u) x = NAN;
    return u & 128u ? -x : x;
}
__device__ __forceinline__ float power(uint32_t b) {
    return b == 255u ? NAN : b ? __uint_as_float(b << 23) : __uint_as_float(0x400000u);
}
__device__ __forceinline__ float operand(const uint8_t* v, int64_t ld, const uint8_t* s, bool t, int64_t i, int64_t n,
                                         int64_t k) {
    const uint32_t b = s[((k / 512) * ((n + 127) / 128) + i / 128) * 512 + (i % 32) * 16 + (i % 128) / 32 * 4 + (k / 128) % 4];
    return decode(t ? v[k * ld + i] : v[i * ld + k]) * power(b);
}

// 64 x 64 outputs per block of 256 threads, 32 of the contracted axis at a time
// through shared memory in fp32.
__global__ void __launch_bounds__(256) matmul_kernel(const MatmulArgs p) {
    __shared__ float as[32][65], bs[32][65];
    const int t = threadIdx.x;
    const int64_t tn = (p.n + 63) / 64;
    const int64_t m0 = blockIdx.x / tn * 64, n0 = blockIdx.x % tn * 64;
    const int ty = t / 16 * 4, tx = t % 16 * 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += 32) {
        for (int e = t; e < 64 * 32; e += 256) {
            const int ia = p.a_t ? e % 64 : e / 32, ka = p.a_t ? e / 64 : e % 32;
            const int ib = p.b_t ? e % 64 : e / 32, kb = p.b_t ? e / 64 : e % 32;
            as[ka][ia] = m0 + ia < p.m && k0 + ka < p.k ? operand(p.a, p.lda, p.sa, p.a_t, m0 + ia, p.m, k0 + ka) : 0.f;
            bs[kb][ib] = n0 + ib < p.n && k0 + kb < p.k ? operand(p.b, p.ldb, p.sb, p.b_t, n0 + ib, p.n, k0 + kb) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 32; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][ty + i], bs[k][tx + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = m0 + ty + i, c = n0 + tx + j;
            if (r >= p.m || c >= p.n) continue;
            const float x = !p.mask || ((p.mask[r * p.wpr + c / 32] >> (c % 32)) & 1u) ? acc[i][j] : 0.f;
            if (p.bf16) {
                uint16_t h;
                asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
                static_cast<uint16_t*>(p.out)[r * p.ldo + c] = h;
            } else {
                static_cast<float*>(p.out)[r * p.ldo + c] = x;
            }
        }
}

}  // namespace
}  // namespace tsenor

using namespace tsenor;

extern "C" tsenor_status tsenor_matmul(tsenor_form form, const uint8_t* a, int64_t lda, const uint8_t* scales_a,
                                       const uint8_t* b, int64_t ldb, const uint8_t* scales_b, int64_t m, int64_t n,
                                       int64_t k, const uint32_t* mask, void* out, tsenor_dtype dtype, int64_t ldo,
                                       tsenor_stream_t stream) {
    if (form != TSENOR_NT && form != TSENOR_NN && form != TSENOR_TN) return TSENOR_ERR_ARG;
    if (dtype != TSENOR_F32 && dtype != TSENOR_BF16) return TSENOR_ERR_ARG;
    const int64_t most = (int64_t(1) << 31) - 1;
    if (m < 0 || n < 0 || k < 0 || m > most || n > most || k > most) return TSENOR_ERR_SHAPE;
    if (((m + 63) / 64) * ((n + 63) / 64) > most) return TSENOR_ERR_SHAPE;
    if (m == 0 || n == 0) return TSENOR_OK;
    const size_t es = dtype == TSENOR_BF16 ? 2 : 4;
    if (!out || !aligned(out, es) || ldo < n || !aligned(mask, 4)) return TSENOR_ERR_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (k == 0) {                            // the empty sum
        const cudaError_t e = cudaMemset2DAsync(out, size_t(ldo) * es, 0, size_t(n) * es, size_t(m), st);
        return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_matmul");
    }
    const bool a_t = form == TSENOR_TN, b_t = form != TSENOR_NT;
    if (!a || !aligned(a, 16) || lda % 16 || lda < (a_t ? m : k) || !b || !aligned(b, 16) || ldb % 16 ||
        ldb < (b_t ? n : k) || !scales_a || !aligned(scales_a, 16) || !scales_b || !aligned(scales_b, 16))
        return TSENOR_ERR_ARG;
    const MatmulArgs p{a, b, lda, ldb, scales_a, scales_b, m, n, k, mask, (n + 31) / 32, out, ldo, a_t, b_t,
                       dtype == TSENOR_BF16};
    matmul_kernel<<<unsigned(((m + 63) / 64) * ((n + 63) / 64)), 256, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_matmul launch");
}
