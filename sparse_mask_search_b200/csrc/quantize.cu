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
// at once).  Row maxima are eight shuffles, column maxima one shuffle and a pass
// through shared memory.  Measured at 4096 x 11008 bf16 (141 MB with the mask) 26 us, 5.4 TB/s, 82 % of the copy rate;
// 88 us while each load was unpacked in the branch that had issued it (one in flight at a time).
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "pdl.h"

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

// 8 entries of a row as they were loaded: 16 bytes of bf16, 32 of fp32.
template <typename T>
struct Eight {
    static constexpr int kWords = sizeof(typename T::storage) * 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const typename T::storage* p) {        // 16-byte aligned
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void load_some(const typename T::storage* p, int64_t n) {     // the first n, the rest 0
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) {
                if constexpr (std::is_same<T, BF16>::value) w[k / 2] |= uint32_t(p[k]) << (16 * (k & 1));
                else w[k] = __float_as_uint(p[k]);
            }
    }
    // The 8 entries at p, of which this thread holds the aligned words from the 16 bytes that p
    // lies in (load_around); the words behind them come from the thread to the right, or, for
    // the last of the 16 threads of a row, from memory.  All threads of the warp take part.
    __device__ __forceinline__ void load_around(const typename T::storage* p) {
        load(reinterpret_cast<const typename T::storage*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15)));
    }
    __device__ __forceinline__ void shift(const typename T::storage* p, bool valid) {
        const unsigned off = unsigned(reinterpret_cast<uintptr_t>(p) & 15u);
        uint4 n = make_uint4(__shfl_down_sync(kFullMask, w[0], 1), __shfl_down_sync(kFullMask, w[1], 1),
                             __shfl_down_sync(kFullMask, w[2], 1), __shfl_down_sync(kFullMask, w[3], 1));
        if ((threadIdx.x & 15) == 15 && valid && off)
            n = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15))[kWords / 4];
        uint32_t u[kWords + 4];
#pragma unroll
        for (int i = 0; i < kWords; ++i) u[i] = w[i];
        u[kWords] = n.x; u[kWords + 1] = n.y; u[kWords + 2] = n.z; u[kWords + 3] = n.w;
#pragma unroll
        for (int i = 0; i + 2 < kWords + 4; ++i) u[i] = off & 8u ? u[i + 2] : u[i];
#pragma unroll
        for (int i = 0; i < kWords + 1; ++i) u[i] = off & 4u ? u[i + 1] : u[i];
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = off & 2u ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
    }
    __device__ __forceinline__ void keep(uint32_t bits) {                        // entries whose bit is 0 become 0
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (std::is_same<T, BF16>::value) {
                const uint32_t b = bits >> (2 * i);
                w[i] &= ((b & 1u) | ((b & 2u) << 15)) * 0xffffu;
            } else {
                w[i] = (bits >> i) & 1u ? w[i] : 0u;
            }
        }
    }
    // A value that is not finite does not take part in its block's maximum: fmaxf drops a
    // NaN, and infinities are made NaN once a thread meets one (rare, so it costs one
    // comparison of the maximum).
    __device__ __forceinline__ void drop_inf() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (std::is_same<T, BF16>::value) {
                if ((w[i] & 0x7fffu) == 0x7f80u) w[i] |= 0x7fffu;
                if ((w[i] & 0x7fff0000u) == 0x7f800000u) w[i] |= 0x7fff0000u;
            } else if ((w[i] & 0x7fffffffu) == 0x7f800000u) {
                w[i] = 0x7fffffffu;
            }
        }
    }
};

// Largest magnitudes of columns, two to a word for bf16 (max.bf16x2 drops a NaN as fmaxf does).
template <typename T>
struct Maxima {
    static constexpr int kWords = Eight<T>::kWords;
    uint32_t w[kWords] = {};

    __device__ __forceinline__ void add(const Eight<T>& v) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (std::is_same<T, BF16>::value)
                asm("max.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(v.w[i] & 0x7fff7fffu), "r"(w[i]));
            else
                w[i] = __float_as_uint(fmaxf(__uint_as_float(w[i]), fabsf(__uint_as_float(v.w[i]))));
        }
    }
    __device__ __forceinline__ float get(int k) const {
        if constexpr (std::is_same<T, BF16>::value)
            return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        else
            return __uint_as_float(w[k]);
    }
    __device__ __forceinline__ float largest() const {
        if constexpr (std::is_same<T, BF16>::value) {
            uint32_t m, n;
            asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w[0]), "r"(w[1]));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(w[2]), "r"(w[3]));
            asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
            return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        } else {
            float m = fmaxf(get(0), get(1));
#pragma unroll
            for (int k = 2; k < 8; ++k) m = fmaxf(m, get(k));
            return m;
        }
    }
};

// Reciprocal scales of 8 columns.  bf16 entries are scaled in bf16: the product with a power of two
// is exact there too, but for results below 2^-126, which round to code 0 all the same.
template <typename T>
struct Scales {
    uint32_t w[Eight<T>::kWords];

    __device__ __forceinline__ void set(int k, float iv) {
        if constexpr (std::is_same<T, BF16>::value) {
            const uint32_t h = __float_as_uint(iv) >> 16;
            w[k / 2] = k & 1 ? w[k / 2] | (h << 16) : h;
        } else {
            w[k] = __float_as_uint(iv);
        }
    }
    __device__ __forceinline__ void set_all(float iv) {
#pragma unroll
        for (int k = 0; k < 8; ++k) set(k, iv);
    }
    // codes of entries 2k and 2k + 1
    __device__ __forceinline__ uint32_t codes(const Eight<T>& v, int k) const {
        if constexpr (std::is_same<T, BF16>::value) {
            uint32_t y;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(v.w[k]), "r"(w[k]));
            return pack2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
        } else {
            return pack2(__uint_as_float(v.w[2 * k]) * __uint_as_float(w[2 * k]),
                         __uint_as_float(v.w[2 * k + 1]) * __uint_as_float(w[2 * k + 1]));
        }
    }
};

// 8 codes of a row, of which the first n lie inside the matrix.
template <typename T>
__device__ __forceinline__ void store8(uint8_t* p, int n, const Eight<T>& v, const Scales<T>& s) {
    const uint32_t lo = s.codes(v, 0) | (s.codes(v, 1) << 16), hi = s.codes(v, 2) | (s.codes(v, 3) << 16);
    if (n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);           // rows start on 16 bytes, columns are a multiple of 8
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) p[k] = uint8_t((k < 4 ? lo >> (8 * k) : hi >> (8 * (k - 4))) & 0xffu);
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
__global__ void __launch_bounds__(kQThreads, sizeof(typename T::storage) == 2 ? 4 : 2) quantize_kernel(const QuantArgs a) {
    __shared__ float part[8][128];          // column maxima of each warp
    __shared__ float colmax[128];
    __shared__ uint8_t rowbyte[128];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t tc = blockIdx.x % a.tiles_c, tr = blockIdx.x / a.tiles_c;
    const int cl = (t & 15) * 8, rl = t >> 4;
    // rows of the tile, and columns from this thread's first one on
    const int rows = a.rows - tr * 128 < 128 ? int(a.rows - tr * 128) : 128;
    const int cols = (a.cols - tc * 128 < 128 ? int(a.cols - tc * 128) : 128) - cl;
    const auto* x = static_cast<const typename T::storage*>(a.x) + (tr * 128 + rl) * a.ldx + tc * 128 + cl;
    const uint8_t* mask = reinterpret_cast<const uint8_t*>(a.mask + (tr * 128 + rl) * a.wpr) + tc * 16 + cl / 8;
    Eight<T> v[kPass];
    uint32_t bits[kPass];
    let_next_start();
    prior_done();
    // A tile with all its columns loads 16 bytes at a time, all in flight together.  Where rows do
    // not start on 16 bytes, the loads cover whole aligned words, up to 15 bytes more on either side, which
    // must not lie outside x: the first tile, and those of the last rows without 8 more columns behind
    // them, go entry by entry, as do tiles that are cut.
    const bool whole = tc * 128 + 128 <= a.cols &&
                       (VEC || (blockIdx.x > 0 && (tr + 1 < a.tiles_r || tc * 128 + 136 <= a.cols)));
    if (whole) {
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            if (rl + 16 * p < rows) {
                if constexpr (VEC) v[p].load(x + 16 * p * a.ldx);
                else v[p].load_around(x + 16 * p * a.ldx);
            } else {
#pragma unroll
                for (int i = 0; i < Eight<T>::kWords; ++i) v[p].w[i] = 0u;
            }
        }
        if constexpr (MASK) {               // 8 columns of a row are one byte of its mask words
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                bits[p] = 0u;
                if (rl + 16 * p < rows) bits[p] = mask[16 * p * a.wpr * 4];
            }
        }
        if constexpr (!VEC) {
#pragma unroll
            for (int p = 0; p < kPass; ++p) v[p].shift(x + 16 * p * a.ldx, rl + 16 * p < rows);
        }
    } else {
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            const int n = rl + 16 * p < rows ? cols : 0;
            v[p].load_some(x + 16 * p * a.ldx, n);
            if constexpr (MASK) bits[p] = n > 0 ? mask[16 * p * a.wpr * 4] : 0u;
        }
    }
    if constexpr (MASK) {                   // a masked entry is 0 whatever it held
#pragma unroll
        for (int p = 0; p < kPass; ++p) v[p].keep(bits[p]);
    }

    uint8_t* out = a.values + (tr * 128 + rl) * a.ldv + tc * 128 + cl;
    Scales<T> by;
    if constexpr (ROW) {
        float m[kPass];
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            Maxima<T> r;
            r.add(v[p]);
            m[p] = r.largest();
            if (m[p] == INFINITY) {
                v[p].drop_inf();
                r = Maxima<T>{};
                r.add(v[p]);
                m[p] = r.largest();
            }
        }
        // The 8 maxima over 16 threads: each exchange halves the rows that a thread carries, so that
        // thread q ends with row q / 2 of its half warp and makes that row's scale for all.
#pragma unroll
        for (int s = 8, n = 4; s >= 2; s >>= 1, n >>= 1)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool high = lane & s;
                const float got = __shfl_xor_sync(kFullMask, high ? m[i] : m[i + n], s);
                m[i] = fmaxf(high ? m[i + n] : m[i], got);
            }
        m[0] = fmaxf(m[0], __shfl_xor_sync(kFullMask, m[0], 1));
        const uint32_t b = scale_byte(m[0]);
        const float iv = inv_scale(b);
        const int mine = rl + 16 * ((t & 15) >> 1);
        if (!(t & 1)) rowbyte[mine] = uint8_t(mine < rows ? b : 127u);
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
            by.set_all(__shfl_sync(kFullMask, iv, (lane & 16) + 2 * p));
            if (rl + 16 * p < rows && cols > 0) store8(out + 16 * p * a.ldv, cols, v[p], by);
        }
        __syncthreads();
        if (t < 128) store_scale(a.scales, a.tiles_r, tr, tc, a.tiles_c, t, rowbyte[t]);
    }
    if constexpr (COL || !ROW) {
        Maxima<T> m;
#pragma unroll
        for (int p = 0; p < kPass; ++p) m.add(v[p]);
        if (m.largest() == INFINITY) {
            m = Maxima<T>{};
#pragma unroll
            for (int p = 0; p < kPass; ++p) {
                v[p].drop_inf();
                m.add(v[p]);
            }
        }
        float w = 0.f;
        if constexpr (COL) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = fmaxf(m.get(k), __shfl_xor_sync(kFullMask, m.get(k), 16));
                if (lane < 16) part[warp][cl + k] = f;
            }
            __syncthreads();
            if (t < 128) {
                w = part[0][t];
#pragma unroll
                for (int k = 1; k < 8; ++k) w = fmaxf(w, part[k][t]);
                colmax[t] = w;
                store_scale(a.scales_t, a.tiles_c, tc, tr, a.tiles_r, t, tc * 128 + t < a.cols ? scale_byte(w) : 127u);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 8; ++k) by.set(k, inv_scale(scale_byte(colmax[cl + k])));
        } else {
            w = m.largest();
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1) w = fmaxf(w, __shfl_xor_sync(kFullMask, w, s));
            if (lane == 0) colmax[warp] = w;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 8; ++k) w = fmaxf(w, colmax[k]);
            const uint32_t b = scale_byte(w);
            by.set_all(inv_scale(b));
            if (t < 128)
                store_scale(a.scales, a.tiles_r, tr, tc, a.tiles_c, t, t < rows ? b : 127u);
            else
                store_scale(a.scales_t, a.tiles_c, tc, tr, a.tiles_r, t - 128, tc * 128 + t - 128 < a.cols ? b : 127u);
        }
        if constexpr (COL) out = a.values_t + (tr * 128 + rl) * a.ldv_t + tc * 128 + cl;
        const int64_t ld = COL ? a.ldv_t : a.ldv;
#pragma unroll
        for (int p = 0; p < kPass; ++p)
            if (rl + 16 * p < rows && cols > 0) store8(out + 16 * p * ld, cols, v[p], by);
    }
}

// Values of the codes: one thread per 4 columns.  The product of a code and a
// power of two is exact in fp32 within its range.
template <typename T>
__global__ void __launch_bounds__(256)
dequantize_kernel(const uint8_t* v, int64_t rows, int64_t cols, int64_t ldv, const uint8_t* scales, bool along_rows,
                  typename T::storage* out, int64_t ldo) {
    const int64_t per = (cols + 3) / 4;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    let_next_start();
    prior_done();
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
    return launch_early(vec ? quantize_kernel<T, ROW, COL, MASK, true> : quantize_kernel<T, ROW, COL, MASK, false>,
                        a.tiles_r * a.tiles_c, kQThreads, 0, 1, st, a);
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
    const cudaError_t e = dtype == TSENOR_BF16
        ? launch_early(dequantize_kernel<BF16>, n, 256, 0, 1, st, values, rows, cols, ldv, scales, along_rows != 0,
                       static_cast<uint16_t*>(out), ldo)
        : launch_early(dequantize_kernel<F32>, n, 256, 0, 1, st, values, rows, cols, ldv, scales, along_rows != 0,
                       static_cast<float*>(out), ldo);
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_dequantize launch");
}
