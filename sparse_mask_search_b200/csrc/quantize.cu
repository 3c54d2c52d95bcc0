// Quantisers of the 8-bit product: e4m3 codes with one power-of-two scale per
// block of 128 entries along a row, of 128 along a column, or of 128 x 128.
//
// Block of entries x with largest finite magnitude a > 0:
//   e = ceil(log2(a / 448)), at least -126;  code = e4m3(x / 2^e)
// 448 is the largest e4m3 value, so no code saturates.  The scale is a power of
// two: x / 2^e is exact in fp32 unless it underflows, so the only rounding of a
// weight or an activation is the one to e4m3 (nearest even, half a step:
// 2^-4 relative), the result is the same on every device, and the tensor cores
// apply the scale themselves, as an exponent byte.
//
// Bound by memory: x is read once (plus one bit per entry with a mask) and one
// byte per entry is written.  One block of 256 threads handles a 128 x 128
// tile, so that row, column and tile maxima all come from one read: sixteen
// threads side by side hold 8 columns each of a row, and a thread holds the same
// 8 columns of 8 rows 16 apart (all eight 16-byte loads are in flight
// at once).  Row maxima are four shuffles, column maxima one shuffle and a pass
// through shared memory.
#include <type_traits>

#include "common.cuh"
#include "host.h"

namespace tsenor {
namespace {

constexpr int kQThreads = 256;
constexpr int kPass = 8;                    // rows of a thread

struct QuantArgs {
    const void* x;
    int64_t rows, cols, ldx;
    const uint32_t* mask;
    int64_t wpr;
    uint8_t* values;                        // row or tile codes
    int64_t ldv;
    uint8_t* values_t;                      // column codes
    int64_t ldv_t;
    uint8_t* scales;
    uint8_t* scales_t;
    int64_t tiles_r, tiles_c;               // ceil(rows / 128), ceil(cols / 128)
};

// Scale byte b (scale 2^(b - 127)) of a block with largest finite magnitude a:
// 448 = 1.75 * 2^8, so the exponent is a's less 8, and one more above 1.75.
__device__ __forceinline__ uint32_t scale_byte(float a) {
    const uint32_t u = __float_as_uint(a);
    const int b = int(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return a > 0.f ? uint32_t(b < 1 ? 1 : b) : 127u;
}
// 1 / 2^(b - 127) for a byte of scale_byte (1 .. 247)
__device__ __forceinline__ float inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two e4m3 codes, round to nearest even; NaN gives 0x7f.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// A value that is not finite does not take part in its block's maximum (fmaxf
// drops a NaN) and gets the NaN code.
__device__ __forceinline__ float drop_inf(float v) { return fabsf(v) == INFINITY ? NAN : v; }

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const QuantArgs& a, int64_t r, int64_t c, float (&v)[8]) {
    const auto* p = static_cast<const typename T::storage*>(a.x) + r * a.ldx + c;
    if (VEC && c + 8 <= a.cols) {
        if constexpr (std::is_same<T, BF16>::value) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
            const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(q[k] << 16);
                v[2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
            }
        } else {
            const float4 w0 = __ldg(reinterpret_cast<const float4*>(p)), w1 = __ldg(reinterpret_cast<const float4*>(p) + 1);
            v[0] = w0.x; v[1] = w0.y; v[2] = w0.z; v[3] = w0.w;
            v[4] = w1.x; v[5] = w1.y; v[6] = w1.z; v[7] = w1.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = 0.f;
            if (c + k < a.cols) {
                if constexpr (std::is_same<T, BF16>::value) v[k] = __uint_as_float(uint32_t(__ldg(p + k)) << 16);
                else v[k] = __ldg(p + k);
            }
        }
    }
}

// 8 codes at column c of a row; only columns inside the matrix are written.
__device__ __forceinline__ void store8(uint8_t* row, int64_t c, int64_t cols, const float (&v)[8], const float (&s)[8]) {
    const uint32_t lo = pack2(v[0] * s[0], v[1] * s[1]) | (pack2(v[2] * s[2], v[3] * s[3]) << 16);
    const uint32_t hi = pack2(v[4] * s[4], v[5] * s[5]) | (pack2(v[6] * s[6], v[7] * s[7]) << 16);
    if (c + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + c) = make_uint2(lo, hi);     // rows start on 16 bytes, c is a multiple of 8
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < cols) row[c + k] = uint8_t((k < 4 ? lo >> (8 * k) : hi >> (8 * (k - 4))) & 0xffu);
    }
}

// Writes the scale bytes of the 128 rows of tile `tile` for block `blk` of the
// contracted axis: byte (r % 32) * 16 + r / 32 * 4 + blk % 4 of the entry
// (blk / 4, tile).  The tile of the last block also fills the entry's unused
// bytes with 127.
__device__ __forceinline__ void store_scale(uint8_t* scales, int64_t tiles, int64_t tile, int64_t blk, int64_t blks,
                                            int r, uint32_t b) {
    uint8_t* p = scales + ((blk / 4) * tiles + tile) * 512 + (r % 32) * 16 + (r / 32) * 4;
    p[blk % 4] = uint8_t(b);
    if (blk == blks - 1)
        for (int64_t k = blk % 4 + 1; k < 4; ++k) p[k] = 127;
}

// ROW: codes and scales of 1 x 128 blocks; COL: of 128 x 1 blocks; neither: 128 x 128.
template <typename T, bool ROW, bool COL, bool MASK, bool VEC>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const QuantArgs a) {
    __shared__ float part[8][128];          // column maxima of each warp
    __shared__ float colmax[128];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t tc = blockIdx.x % a.tiles_c, tr = blockIdx.x / a.tiles_c;
    const int cl = (t & 15) * 8, rl = t >> 4;
    const int64_t c = tc * 128 + cl, r0 = tr * 128 + rl;
    float v[kPass][8];
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
        const int64_t r = r0 + 16 * p;
        if (r < a.rows && c < a.cols) {
            load8<T, VEC>(a, r, c, v[p]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[p][k] = 0.f;
        }
    }
    if constexpr (MASK) {
        // 8 columns of a row are one byte of its mask words; a masked entry is 0 whatever it held
        uint32_t m[kPass];
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const int64_t r = r0 + 16 * p;
            m[p] = r < a.rows && c < a.cols ? reinterpret_cast<const uint8_t*>(a.mask + r * a.wpr)[c / 8] : 0u;
        }
#pragma unroll
        for (int p = 0; p < kPass; ++p)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[p][k] = (m[p] >> k) & 1u ? v[p][k] : 0.f;
    }
#pragma unroll
    for (int p = 0; p < kPass; ++p)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[p][k] = drop_inf(v[p][k]);

    if constexpr (ROW) {
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[p][k]));
#pragma unroll
            for (int s = 8; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, s));
            const uint32_t b = scale_byte(m);
            const float iv = inv_scale(b);
            const float s[8] = {iv, iv, iv, iv, iv, iv, iv, iv};
            const int64_t r = r0 + 16 * p;
            if (r < a.rows && c < a.cols) store8(a.values + r * a.ldv, c, a.cols, v[p], s);
            if ((t & 15) == 0) store_scale(a.scales, a.tiles_r, tr, tc, a.tiles_c, rl + 16 * p, r < a.rows ? b : 127u);
        }
    }
    if constexpr (COL || !ROW) {
        float m[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] = 0.f;
#pragma unroll
            for (int p = 0; p < kPass; ++p) m[k] = fmaxf(m[k], fabsf(v[p][k]));
            m[k] = fmaxf(m[k], __shfl_xor_sync(kFullMask, m[k], 16));
        }
        if (lane < 16) {
#pragma unroll
            for (int k = 0; k < 8; ++k) part[warp][cl + k] = m[k];
        }
        __syncthreads();
        if (t < 128) {
            float w = part[0][t];
#pragma unroll
            for (int k = 1; k < 8; ++k) w = fmaxf(w, part[k][t]);
            if constexpr (!COL) {
#pragma unroll
                for (int s = 16; s >= 1; s >>= 1) w = fmaxf(w, __shfl_xor_sync(kFullMask, w, s));
            }
            colmax[t] = w;
        }
        __syncthreads();
        float s[8];
        if constexpr (COL) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = inv_scale(scale_byte(colmax[cl + k]));
            if (t < 128)
                store_scale(a.scales_t, a.tiles_c, tc, tr, a.tiles_r, t,
                            tc * 128 + t < a.cols ? scale_byte(colmax[t]) : 127u);
        } else {
            const uint32_t b = scale_byte(fmaxf(fmaxf(colmax[0], colmax[32]), fmaxf(colmax[64], colmax[96])));
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = inv_scale(b);
            if (t < 128)
                store_scale(a.scales, a.tiles_r, tr, tc, a.tiles_c, t, tr * 128 + t < a.rows ? b : 127u);
            else
                store_scale(a.scales_t, a.tiles_c, tc, tr, a.tiles_r, t - 128, tc * 128 + t - 128 < a.cols ? b : 127u);
        }
        uint8_t* out = COL ? a.values_t : a.values;
        const int64_t ld = COL ? a.ldv_t : a.ldv;
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const int64_t r = r0 + 16 * p;
            if (r < a.rows && c < a.cols) store8(out + r * ld, c, a.cols, v[p], s);
        }
    }
}

// Values of the codes: one thread per 4 columns.  The product of a code and a
// power of two is exact in fp32 within its range.
template <typename T>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint8_t* __restrict__ v, int64_t rows, int64_t cols, int64_t ldv,
                  const uint8_t* __restrict__ scales, bool along_rows, typename T::storage* __restrict__ out, int64_t ldo) {
    const int64_t per = (cols + 3) / 4;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= rows * per) return;
    const int64_t r = i / per, c0 = i % per * 4;
    const int64_t tiles = ((along_rows ? cols : rows) + 127) / 128;
    for (int k = 0; k < 4 && c0 + k < cols; ++k) {
        const int64_t c = c0 + k, o = along_rows ? c : r, in = along_rows ? r : c;
        const uint32_t b = scales[((in / 512) * tiles + o / 128) * 512 + (o % 32) * 16 + (o % 128) / 32 * 4 + (in / 128) % 4];
        const uint32_t u = v[r * ldv + c], e = (u >> 3) & 15u, f = u & 7u;
        float x = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : float(f) * 0.001953125f;
        if ((u & 127u) == 127u) x = NAN;
        x = u & 128u ? -x : x;
        // 2^(b - 127): b = 0 is a subnormal, 255 stands for NaN
        x *= b == 255u ? NAN : b ? __uint_as_float(b << 23) : __uint_as_float(0x400000u);
        if constexpr (std::is_same<T, BF16>::value) {
            uint16_t h;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
            out[r * ldo + c] = h;
        } else {
            out[r * ldo + c] = x;
        }
    }
}

template <typename T, bool ROW, bool COL, bool MASK>
cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t st) {
    constexpr int es = sizeof(typename T::storage);
    const bool vec = aligned(a.x, 16) && (a.rows == 1 || a.ldx * es % 16 == 0);
    const unsigned grid = unsigned(a.tiles_r * a.tiles_c);
    if (vec) quantize_kernel<T, ROW, COL, MASK, true><<<grid, kQThreads, 0, st>>>(a);
    else quantize_kernel<T, ROW, COL, MASK, false><<<grid, kQThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <bool ROW, bool COL>
cudaError_t dispatch_quantize(tsenor_dtype dtype, const QuantArgs& a, cudaStream_t st) {
    if constexpr (!(ROW && COL)) {          // the pair has no mask
        if (a.mask)
            return dtype == TSENOR_BF16 ? launch_quantize<BF16, ROW, COL, true>(a, st)
                                        : launch_quantize<F32, ROW, COL, true>(a, st);
    }
    return dtype == TSENOR_BF16 ? launch_quantize<BF16, ROW, COL, false>(a, st)
                                : launch_quantize<F32, ROW, COL, false>(a, st);
}

tsenor_status check_matrix(int dtype, int64_t rows, int64_t cols) {
    if (dtype != TSENOR_F32 && dtype != TSENOR_BF16) return TSENOR_ERR_ARG;
    if (rows < 0 || cols < 0 || rows > (int64_t(1) << 31) - 1 || cols > (int64_t(1) << 31) - 1) return TSENOR_ERR_SHAPE;
    if (((rows + 127) / 128) * ((cols + 127) / 128) > (int64_t(1) << 31) - 1) return TSENOR_ERR_SHAPE;
    return TSENOR_OK;
}

bool codes_ok(const uint8_t* values, int64_t ldv, int64_t cols) {
    return values && aligned(values, 16) && ldv >= cols && ldv % 16 == 0;
}

bool input_ok(const void* x, int dtype, int64_t ldx, int64_t cols) {
    return x && aligned(x, dtype == TSENOR_BF16 ? 2 : 4) && ldx >= cols;
}

}  // namespace
}  // namespace tsenor

using namespace tsenor;

extern "C" int64_t tsenor_scale_bytes(int64_t rows, int64_t cols) {
    return rows < 1 || cols < 1 ? 0 : ((cols + 511) / 512) * ((rows + 127) / 128) * 512;
}

extern "C" tsenor_status tsenor_quantize(const void* x, tsenor_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                         tsenor_block block, const uint32_t* mask, uint8_t* values, int64_t ldv,
                                         uint8_t* scales, uint8_t* scales_t, tsenor_stream_t stream) {
    const tsenor_status s = check_matrix(dtype, rows, cols);
    if (s != TSENOR_OK) return s;
    if (block != TSENOR_BLOCK_ROW && block != TSENOR_BLOCK_COLUMN && block != TSENOR_BLOCK_TILE) return TSENOR_ERR_ARG;
    if (rows == 0 || cols == 0) return TSENOR_OK;
    if (!input_ok(x, dtype, ldx, cols) || !codes_ok(values, ldv, cols) || !aligned(mask, 4)) return TSENOR_ERR_ARG;
    if (block != TSENOR_BLOCK_COLUMN && (!scales || !aligned(scales, 16))) return TSENOR_ERR_ARG;
    if (block != TSENOR_BLOCK_ROW && (!scales_t || !aligned(scales_t, 16))) return TSENOR_ERR_ARG;
    QuantArgs a{x, rows, cols, ldx, mask, (cols + 31) / 32, values, ldv, values, ldv, scales, scales_t,
                (rows + 127) / 128, (cols + 127) / 128};
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = block == TSENOR_BLOCK_ROW      ? dispatch_quantize<true, false>(dtype, a, st)
                          : block == TSENOR_BLOCK_COLUMN ? dispatch_quantize<false, true>(dtype, a, st)
                                                         : dispatch_quantize<false, false>(dtype, a, st);
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_quantize launch");
}

extern "C" tsenor_status tsenor_quantize_pair(const void* x, tsenor_dtype dtype, int64_t rows, int64_t cols, int64_t ldx,
                                              uint8_t* values, int64_t ldv, uint8_t* scales, uint8_t* values_t,
                                              int64_t ldv_t, uint8_t* scales_t, tsenor_stream_t stream) {
    const tsenor_status s = check_matrix(dtype, rows, cols);
    if (s != TSENOR_OK) return s;
    if (rows == 0 || cols == 0) return TSENOR_OK;
    if (!input_ok(x, dtype, ldx, cols) || !codes_ok(values, ldv, cols) || !codes_ok(values_t, ldv_t, cols) ||
        values == values_t || !scales || !aligned(scales, 16) || !scales_t || !aligned(scales_t, 16))
        return TSENOR_ERR_ARG;
    QuantArgs a{x, rows, cols, ldx, nullptr, 0, values, ldv, values_t, ldv_t, scales, scales_t,
                (rows + 127) / 128, (cols + 127) / 128};
    const cudaError_t e = dispatch_quantize<true, true>(dtype, a, (cudaStream_t)stream);
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_quantize_pair launch");
}

extern "C" tsenor_status tsenor_dequantize(const uint8_t* values, int64_t rows, int64_t cols, int64_t ldv,
                                           const uint8_t* scales, int along_rows, void* out, tsenor_dtype dtype,
                                           int64_t ldo, tsenor_stream_t stream) {
    const tsenor_status s = check_matrix(dtype, rows, cols);
    if (s != TSENOR_OK) return s;
    if (rows == 0 || cols == 0) return TSENOR_OK;
    if (!values || ldv < cols || !scales || !input_ok(out, dtype, ldo, cols)) return TSENOR_ERR_ARG;
    const int64_t n = (rows * ((cols + 3) / 4) + 255) / 256;
    if (n > (int64_t(1) << 31) - 1) return TSENOR_ERR_SHAPE;
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == TSENOR_BF16)
        dequantize_kernel<BF16><<<unsigned(n), 256, 0, st>>>(values, rows, cols, ldv, scales, along_rows != 0,
                                                             static_cast<uint16_t*>(out), ldo);
    else
        dequantize_kernel<F32><<<unsigned(n), 256, 0, st>>>(values, rows, cols, ldv, scales, along_rows != 0,
                                                            static_cast<float*>(out), ldo);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_dequantize launch");
}
