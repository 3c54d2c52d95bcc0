// Product of two e4m3 matrices with a power-of-two scale per block of 128 along
// the contracted axis:
//   nt  out[m,n] = sum_k A[m,k] B[n,k]     nn  A[m,k] B[k,n]     tn  A[k,m] B[k,n]
//
// The scales are exponents, so the tensor cores apply them (kind::mxf8f6f4, one byte per row and 32 of the
// contracted axis; the same byte for four such steps): sums stay in tensor memory in fp32 from the first block to
// the last and are rounded once.  What they lose on the way is the instruction's: it cuts the 32 products and the sum below
// 2^-25 of the largest of them (11008 x 4096 x 2048 on activations: 1.6e-7 of the result's norm, 0.7e-7 with every addition
// rounded), which more accumulators and additions outside the tensor cores would lessen at the price of a pass for each.
// Codes stored along either axis are read as they are, K-major or MN-major.
// Bound by the tensor cores (and, on random data, by the card's power limit) for many rows, by the bytes
// of B for few.  Measured, with the host's share: 4096 x 28672 x 8192 nt 757 us (2.54 PFLOP/s; 486 us on zeros, where
// the clock stays at 1965 MHz), 2048 x 11008 x 4096 84 us, 1 x 11008 x 4096 12.3 us (3.7 TB/s).
#include <mutex>

#include <cudaTypedefs.h>

#include "common.cuh"
#include "host.h"
#include "pdl.h"
#include "tensor.h"

namespace tsenor {
namespace {

struct MatmulArgs {
    const uint8_t *sa, *sb;
    int64_t m, n, k;
    const uint32_t* mask;
    int64_t wpr;
    void* out;
    int64_t ldo;
    int64_t tiles_m, tiles_n;   // of 128
    int a_bytes;                // bytes that one TMA copy of an A tile writes
    int stages;
    bool a_t, b_t;              // the operand is stored with its contracted axis along rows
    bool bf16;
    bool vec;                   // rows of the output are aligned to the kernel's vector stores
};

__device__ unsigned long long g_stalled;

constexpr int kTile = 128;                       // rows, columns and summed entries of a tile
constexpr int kTileBytes = kTile * kTile;
constexpr int kScaleBytes = 512;
constexpr int kSms = 148;                        // of a B200: grids and the choice of a kernel are made for it
constexpr int kPad = 132;                        // floats to a staged row: 16-byte stores without bank conflicts

// An epilogue waits for as long as a tile's sums take: the bound grows with their number.
__device__ __forceinline__ bool wait_long(uint64_t* bar, unsigned parity, int64_t blocks) {
    for (int64_t i = 0; i <= blocks / 64; ++i)
        if (warp_sleep(bar, parity)) return true;
    return false;
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
}

// Four sums of row r from column c on: mask, rounding, store.
template <bool BF16OUT>
__device__ __forceinline__ void store4(const MatmulArgs& p, int64_t r, int64_t c, float4 v) {
    float x[4] = {v.x, v.y, v.z, v.w};
    if (p.mask) {
        const uint32_t w = p.mask[r * p.wpr + c / 32] >> (c % 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (w >> i) & 1u ? x[i] : 0.f;
    }
    if constexpr (BF16OUT) {
        uint16_t* o = static_cast<uint16_t*>(p.out) + r * p.ldo + c;
        if (p.vec && c + 4 <= p.n) {
            *reinterpret_cast<uint2*>(o) = make_uint2(to_bf16(x[0]) | (uint32_t(to_bf16(x[1])) << 16),
                                                      to_bf16(x[2]) | (uint32_t(to_bf16(x[3])) << 16));
        } else {
            for (int i = 0; i < 4; ++i)
                if (c + i < p.n) o[i] = to_bf16(x[i]);
        }
    } else {
        float* o = static_cast<float*>(p.out) + r * p.ldo + c;
        if (p.vec && c + 4 <= p.n) {
            *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
            for (int i = 0; i < 4; ++i)
                if (c + i < p.n) o[i] = x[i];
        }
    }
}

// Mask words of a row for 128 columns from c on; asked for before the sums are ready.
__device__ __forceinline__ void load_mask(const MatmulArgs& p, int64_t r, int64_t c, uint32_t (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = p.mask && r < p.m && c + 32 * i < p.n ? p.mask[r * p.wpr + c / 32 + i] : 0xffffffffu;
}
__device__ __forceinline__ void apply_mask(uint32_t w, uint32_t (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = (w >> i) & 1u ? v[i] : 0u;
}

// 32 sums of row r from column c on, held by one thread.
template <bool BF16OUT>
__device__ __forceinline__ void store_row(const MatmulArgs& p, int64_t r, int64_t c, const uint32_t (&v)[32]) {
    if constexpr (BF16OUT) {
        uint16_t* o = static_cast<uint16_t*>(p.out) + r * p.ldo + c;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[i])
                    : "f"(__uint_as_float(v[16 * q + 2 * i + 1])), "f"(__uint_as_float(v[16 * q + 2 * i])));
            if (c + 16 * q + 16 <= p.n) {
                store32(o + 16 * q, h);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + 16 * q + i < p.n) o[16 * q + i] = uint16_t(i & 1 ? h[i / 2] >> 16 : h[i / 2] & 0xffffu);
            }
        }
    } else {
        float* o = static_cast<float*>(p.out) + r * p.ldo + c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (c + 8 * q + 8 <= p.n) {
                uint32_t h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = v[8 * q + i];
                store32(o + 8 * q, h);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + 8 * q + i < p.n) o[8 * q + i] = __uint_as_float(v[8 * q + i]);
            }
        }
    }
}

// The same for rows that do not start on 32 bytes: the warp's 32 x 32 sums turn
// through shared memory, so that a store instruction covers one row.  Where the product is short this
// bounds the call: 2899 x 16023 x 20 tn to bf16 91 us (113 with one row's load and store after another), 30 us with 16032
// columns or an output whose rows start on 32 bytes.
template <bool BF16OUT>
__device__ __forceinline__ void store_turned(const MatmulArgs& p, int64_t r0, int64_t c, const uint32_t (&v)[32], float* staged) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) staged[lane * 33 + i] = __uint_as_float(v[i]);
    __syncwarp();
    if (c + lane >= p.n) return;
    const int rows = p.m - r0 < 32 ? int(p.m - r0) : 32;
    const int64_t at = r0 * p.ldo + c + lane;
    constexpr int kAhead = 8;                    // the loads of eight rows before their stores
    for (int i = 0; i < rows; i += kAhead) {
        float x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) x[k] = staged[(i + k) * 33 + lane];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + k >= rows) break;
            if constexpr (BF16OUT) static_cast<uint16_t*>(p.out)[at + (i + k) * p.ldo] = to_bf16(x[k]);
            else static_cast<float*>(p.out)[at + (i + k) * p.ldo] = x[k];
        }
    }
}

// ---- few rows, or few tiles --------------------------------------------------------------
//
// 128 x 128 tiles.  Warp 0 loads (TMA, a ring of stages), warp 1 issues the products,
// warps 2 to 5 store.  A kernel that holds tensor memory runs one CTA to an SM, so a CTA takes all
// of its shared memory: what bounds a product of few rows is the bytes of B in flight.
//
// SPLIT: a tile belongs to a cluster of `split` CTAs; each sums its share of the blocks
// of 128, and the shares are added in rank order through distributed shared memory.
// Otherwise the CTAs are persistent and walk the tiles, with two accumulators, so that the
// loads of the next tile never wait for a store.
constexpr int kThreads = 192;
constexpr int kTmemCols = 512;                   // two accumulators of 128, 4 columns of each side's scales
constexpr int kStageBytes = 224 * 1024;          // of all stages and the room to turn

// Shared memory from its 1024-byte aligned base: the A tiles (which may be shorter than
// 128 rows: the rows behind them are read by the tensor core and go to rows of the
// accumulator that nothing reads), the B tiles, the scales, room to turn 32 x 32 sums, the barriers.
// The shares of a split tile are staged over the tiles at the end.
struct TileSmem {
    unsigned a, b, s, turn, bars;
    __host__ __device__ TileSmem(int stages, int a_bytes) {
        a = 0;
        b = stages * a_bytes;
        s = b + stages * kTileBytes;
        turn = s + stages * 2 * kScaleBytes;
        bars = turn + 4 * 32 * 33 * 4;
    }
    __host__ __device__ unsigned bytes(int stages) const { return bars + (2 * stages + 5) * 8 + 16; }
};
// The most that a launch asks for: the smallest stage (8 rows of A) gives 12 stages at most.
constexpr unsigned kTileMost = kStageBytes + (2 * (kStageBytes / (9 * 1024 * 2)) + 5) * 8 + 16 + 1024;
static_assert(kTileMost <= 227 * 1024, "shared memory of a CTA");

template <bool SPLIT, bool BF16OUT>
__global__ void __launch_bounds__(kThreads, 1)
tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const MatmulArgs p,
            const int split) {
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const TileSmem at(p.stages, p.a_bytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + at.bars);
    uint64_t* empty = full + p.stages;
    uint64_t* ready = empty + p.stages;          // an accumulator is complete
    uint64_t* room = ready + 2;                  // an accumulator has been read
    uint64_t* over = room + 2;                   // no product is in flight any more
    uint32_t* slot = reinterpret_cast<uint32_t*>(over + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = SPLIT ? cluster_rank() : 0;
    const int64_t tiles = p.tiles_m * p.tiles_n, blocks = (p.k + kTile - 1) / kTile;
    const int64_t first = SPLIT ? blockIdx.x / split : blockIdx.x, step = SPLIT ? tiles : gridDim.x;
    const int64_t k0 = SPLIT ? blocks * rank / split : 0, k1 = SPLIT ? blocks * (rank + 1) / split : blocks;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(ready + i, 1);
            mbar_init(room + i, 4);
        }
        mbar_init(over, 1);
        mbar_init_fence();
    }
    let_next_start();
    __syncthreads();
    if (warp != 1) prior_done();
    bool stalled = false;

    if (warp == 0) {                             // loads start while warp 1 gets its tensor memory
        int st = 0;
        unsigned phase = 0;
        bool around = false;                     // every stage has been used
        for (int64_t t = first; t < tiles && !stalled; t += step) {
            const int64_t tm = t % p.tiles_m, tn = t / p.tiles_m;
            const int m = int(tm * kTile), n = int(tn * kTile);
            for (int64_t kb = k0; kb < k1; ++kb) {
                if (!warp_wait(empty + st, phase ^ 1)) { stalled = true; break; }
                if (elect_one()) {
                    const bool scales = kb == k0 || kb % 4 == 0;
                    mbar_arrive_expect_tx(full + st, p.a_bytes + kTileBytes + (scales ? 2 * kScaleBytes : 0));
                    const int k = int(kb * kTile);
                    tma_load_2d(smem + at.a + st * p.a_bytes, &map_a, p.a_t ? m : k, p.a_t ? k : m, full + st);
                    tma_load_2d(smem + at.b + st * kTileBytes, &map_b, p.b_t ? n : k, p.b_t ? k : n, full + st);
                    if (scales) {
                        uint8_t* d = smem + at.s + st * 2 * kScaleBytes;
                        bulk_load(d, p.sa + ((kb / 4) * p.tiles_m + tm) * kScaleBytes, kScaleBytes, full + st);
                        bulk_load(d + kScaleBytes, p.sb + ((kb / 4) * p.tiles_n + tn) * kScaleBytes, kScaleBytes, full + st);
                    }
                }
                __syncwarp();
                if (++st == p.stages) { st = 0; phase ^= 1; around = true; }
            }
        }
        // copies in flight end before the block does, whichever warp gave up
        for (int i = 0; i < p.stages; ++i)
            if ((around || i < st) && !warp_drain(full + i, i < st ? phase : phase ^ 1)) stalled = true;
    } else if (warp == 1) {
        const uint32_t idesc = mma_desc(kTile, kTile, p.a_t, p.b_t);
        // 32 of the contracted axis: 32 bytes of a row, or 32 rows
        const uint32_t step_a = (p.a_t ? 4096 : 32) >> 4, step_b = (p.b_t ? 4096 : 32) >> 4;
        tmem_alloc<1>(slot, kTmemCols);
        prior_done();                            // no limited wait counts the time of the kernel before
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(slot), ts = tmem + 2 * kTile;
        int st = 0;
        unsigned phase = 0, n = 0;
        for (int64_t t = first; t < tiles && !stalled; t += step, ++n) {
            if (n > 1 && !warp_wait(room + (n & 1), ((n >> 1) - 1) & 1)) { stalled = true; break; }
            tmem_fence_after();
            const uint32_t d = tmem + (n & 1) * kTile;
            for (int64_t kb = k0; kb < k1; ++kb) {
                if (!warp_wait(full + st, phase)) { stalled = true; break; }
                tmem_fence_after();
                if (elect_one()) {
                    if (kb == k0 || kb % 4 == 0) {
                        const uint32_t s = smem_u32(smem + at.s + st * 2 * kScaleBytes);
                        copy_scales<1>(ts, scale_desc(s));
                        copy_scales<1>(ts + 4, scale_desc(s + kScaleBytes));
                    }
                    const uint32_t id = with_scale_byte(idesc, uint32_t(kb % 4));
                    const uint64_t da = tile_desc(smem_u32(smem + at.a + st * p.a_bytes), kTileBytes);
                    const uint64_t db = tile_desc(smem_u32(smem + at.b + st * kTileBytes), kTileBytes);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_scaled<1>(d, da + i * step_a, db + i * step_b, id, ts, ts + 4, kb > k0 || i > 0);
                    mma_commit(empty + st);
                }
                __syncwarp();
                if (++st == p.stages) { st = 0; phase ^= 1; }
            }
            if (!stalled && elect_one()) mma_commit(ready + (n & 1));
            __syncwarp();
        }
        // products in flight end before their tiles and tensor memory go, whichever warp gave up
        if (elect_one()) mma_commit(over);
        __syncwarp();
        if (!warp_drain(over, 0)) stalled = true;
    } else {
        const int quarter = warp & 3;            // the lanes of tensor memory that a warp may read
        float* turn = reinterpret_cast<float*>(smem + at.turn) + quarter * 32 * 33;
        float* staged = reinterpret_cast<float*>(smem);
        unsigned n = 0;
        for (int64_t t = first; t < tiles; t += step, ++n) {
            const int64_t r0 = t % p.tiles_m * kTile + quarter * 32, c0 = t / p.tiles_m * kTile;
            uint32_t mask[4];
            if constexpr (!SPLIT) load_mask(p, r0 + lane, c0, mask);
            if (!wait_long(ready + (n & 1), (n >> 1) & 1, k1 - k0)) { stalled = true; break; }
            tmem_fence_after();
            const uint32_t d = *reinterpret_cast<volatile uint32_t*>(slot) + (uint32_t(quarter * 32) << 16) + (n & 1) * kTile;
            if (r0 < p.m) {
#pragma unroll
                for (int c = 0; c < kTile; c += 32) {
                    uint32_t v[32];
                    tmem_load32(d + c, v);
                    tmem_wait_load(v);
                    if constexpr (SPLIT) {
                        if (r0 + lane < p.m) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<uint4*>(staged + (quarter * 32 + lane) * kPad + c + i) =
                                    make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        }
                    } else if (c0 + c < p.n) {
                        apply_mask(mask[c / 32], v);
                        if (p.vec) {
                            if (r0 + lane < p.m) store_row<BF16OUT>(p, r0 + lane, c0 + c, v);
                        } else {
                            store_turned<BF16OUT>(p, r0, c0 + c, v, turn);
                        }
                    }
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(room + (n & 1));
        }
    }
    if (stalled && lane == 0) atomicAdd(&g_stalled, 1ull);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 1) tmem_free<1>(*slot, kTmemCols);
    if constexpr (SPLIT) {
        cluster_sync();
        const int64_t tm = first % p.tiles_m, tn = first / p.tiles_m;
        const int rows = int(p.m - tm * kTile < kTile ? p.m - tm * kTile : kTile);
        const uint32_t base = smem_u32(smem);
        // four sums of four columns at a time, so that their loads are in flight together
        constexpr int kAhead = 4;
        const int units = rows * (kTile / 4), step_u = split * kThreads;
        for (int u0 = int(rank) * kThreads + threadIdx.x; u0 < units; u0 += kAhead * step_u) {
            float4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q = 0; q < split; ++q) {
                float4 w[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int u = u0 + i * step_u;
                    if (u < units)
                        w[i] = cluster_load4(cluster_addr(base + (u / (kTile / 4) * kPad + u % (kTile / 4) * 4) * 4, q));
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (u0 + i * step_u < units)
                        v[i] = make_float4(v[i].x + w[i].x, v[i].y + w[i].y, v[i].z + w[i].z, v[i].w + w[i].w);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int u = u0 + i * step_u;
                const int r = u / (kTile / 4), c = u % (kTile / 4) * 4;
                if (u < units && tn * kTile + c < p.n) store4<BF16OUT>(p, tm * kTile + r, tn * kTile + c, v[i]);
            }
        }
        cluster_sync();                          // a peer's shared memory lives until all have read it
    }
}

// ---- large products -------------------------------------------------------------------
//
// A pair of CTAs works on a 256 x 256 tile (cta_group::2): each holds 128 rows of
// A and 128 of B in shared memory and 128 rows of the accumulator.  The pairs are
// persistent.  Two accumulators of 256 columns and the scales do not fit into
// 512 columns of tensor memory, so the second one starts at column 240: its
// product may start once the 32 columns that hold the overlap have been read, which
// the epilogue does first.  A 256 x 256 tile, because each byte that an SM takes in is used by one product only:
// at 128 x 128 the loads alone (64 bytes a cycle and SM) took twice the products' time, here they take as long.
// Between the two kernels the fitted costs at `launch` decide.  Five stages are what shared memory holds; with four
// 2048 x 11008 x 4096 takes 76.5 us where it takes 72.0 (on one card).
constexpr int kPairThreads = 384;                // warps: 0 loads, 1 products, 2 tensor memory, 4 to 11 epilogue
constexpr int kPairTile = 256;
constexpr int kPairStages = 5;
constexpr int kSecond = 240, kScaleA = 496, kScaleB = 500;
constexpr int kGroupM = 16;                      // tiles of 256 rows walked together, so that B is read from L2

struct PairSmem {
    static constexpr unsigned a = 0, b = kPairStages * kTileBytes, s = 2 * b, staged = s + kPairStages * 3 * kScaleBytes,
                              bars = staged + 8 * 32 * 33 * 4, bytes = bars + (2 * kPairStages + 4) * 8 + 2 * 8 + 2 * 4;
};

// Tile t of the walk: groups of kGroupM tile rows, column by column within a group.
__device__ __forceinline__ void pair_tile(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t* tm, int64_t* tn) {
    const int64_t group = t / (kGroupM * tiles_n), first = group * kGroupM;
    const int64_t height = tiles_m - first < kGroupM ? tiles_m - first : kGroupM;
    const int64_t in = t - group * kGroupM * tiles_n;
    *tm = first + in % height;
    *tn = in / height;
}

template <bool BF16OUT>
__global__ void __launch_bounds__(kPairThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb, const MatmulArgs p) {
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + PairSmem::bars);
    uint64_t* empty = full + kPairStages;
    uint64_t* ready = empty + kPairStages;       // an accumulator is complete (one barrier for each of the two)
    uint64_t* room = ready + 2;                  // the next accumulator may be written
    uint64_t* over = room + 1;                   // no product is in flight any more
    int64_t* issued = reinterpret_cast<int64_t*>(over + 1);      // stages that each CTA's copies went to; in rank 0
    uint32_t* slot = reinterpret_cast<uint32_t*>(issued + 2);
    uint32_t* gave_up = slot + 1;                // some warp of the pair
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned rank = cluster_rank();
    const int64_t tiles_m = (p.m + kPairTile - 1) / kPairTile, tiles_n = (p.n + kPairTile - 1) / kPairTile;
    const int64_t tiles = tiles_m * tiles_n, blocks = (p.k + kTile - 1) / kTile;
    const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(full + i, 1);              // used in the CTA of rank 0, which expects both CTAs' bytes
            mbar_init(empty + i, 1);
        }
        mbar_init(ready, 1);
        mbar_init(ready + 1, 1);
        mbar_init(room, 16);                     // the epilogue warps of both CTAs; used in rank 0
        mbar_init(over, 1);
        *gave_up = 0;
        mbar_init_fence();
    }
    if (warp == 2) tmem_alloc<2>(slot, 512);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = *slot;
    let_next_start();
    if (warp != 1) prior_done();
    bool stalled = false;

    if (warp == 0) {
        // A stage of rank 0's CTA is full when the bytes of both CTAs are there.  Rank 1's copies may
        // count before rank 0 expects them: the stage was free in both CTAs, so its barrier is
        // already in this phase, and the phase cannot end without rank 0's arrival.
        const uint32_t full0 = cluster_addr(smem_u32(full), 0);
        int st = 0;
        unsigned phase = 0;
        int64_t count = 0;
        for (int64_t t = first; t < tiles && !stalled; t += step) {
            int64_t tm, tn;
            pair_tile(t, tiles_m, tiles_n, &tm, &tn);
            const int64_t a128 = tm * 2 + rank, b128 = tn * 2 + rank;
            const int m = int(a128 * kTile), n = int(b128 * kTile);
            for (int64_t kb = 0; kb < blocks; ++kb) {
                if (!warp_wait(empty + st, phase ^ 1)) { stalled = true; break; }
                if (elect_one()) {
                    const uint32_t bar = full0 + st * 8;
                    if (rank == 0) mbar_arrive_expect_tx(full + st, 4 * kTileBytes + (kb % 4 == 0 ? 6 * kScaleBytes : 0));
                    const int k = int(kb * kTile);
                    tma_load_pair(smem + PairSmem::a + st * kTileBytes, &map_a, p.a_t ? m : k, p.a_t ? k : m, bar);
                    tma_load_pair(smem + PairSmem::b + st * kTileBytes, &map_b, p.b_t ? n : k, p.b_t ? k : n, bar);
                    if (kb % 4 == 0) {
                        uint8_t* d = smem + PairSmem::s + st * 3 * kScaleBytes;
                        tma_load_pair(d, &map_sa, 0, int((kb / 4) * p.tiles_m + a128), bar);
                        tma_load_pair(d + kScaleBytes, &map_sb, 0, int((kb / 4) * p.tiles_n + tn * 2), bar);
                    }
                }
                __syncwarp();
                ++count;
                if (++st == kPairStages) { st = 0; phase ^= 1; }
            }
        }
        if (lane == 0) cluster_store(cluster_addr(smem_u32(issued + rank), 0), count);
    } else if (warp == 1 && rank == 0) {
        prior_done();                            // no limited wait counts the time of the kernel before
        const uint32_t idesc = mma_desc(kPairTile, kPairTile, p.a_t, p.b_t);
        const uint32_t step_a = (p.a_t ? 4096 : 32) >> 4, step_b = (p.b_t ? 4096 : 32) >> 4;
        int st = 0;
        unsigned phase = 0, n = 0;
        for (int64_t t = first; t < tiles && !stalled; t += step, ++n) {
            if (n > 0 && !warp_wait(room, (n - 1) & 1)) { stalled = true; break; }
            tmem_fence_after();
            const uint32_t d = tmem + (n & 1 ? kSecond : 0);
            for (int64_t kb = 0; kb < blocks; ++kb) {
                if (!warp_wait(full + st, phase)) { stalled = true; break; }
                tmem_fence_after();
                if (elect_one()) {
                    if (kb % 4 == 0) {
                        const uint32_t s = smem_u32(smem + PairSmem::s + st * 3 * kScaleBytes);
                        copy_scales<2>(tmem + kScaleA, scale_desc(s));
                        copy_scales<2>(tmem + kScaleB, scale_desc(s + kScaleBytes));
                        copy_scales<2>(tmem + kScaleB + 4, scale_desc(s + 2 * kScaleBytes));
                    }
                    const uint32_t id = with_scale_byte(idesc, uint32_t(kb % 4));
                    const uint64_t da = tile_desc(smem_u32(smem + PairSmem::a + st * kTileBytes), kTileBytes);
                    const uint64_t db = tile_desc(smem_u32(smem + PairSmem::b + st * kTileBytes), kTileBytes);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_scaled<2>(d, da + i * step_a, db + i * step_b, id, tmem + kScaleA, tmem + kScaleB, kb > 0 || i > 0);
                    mma_commit_pair(empty + st);
                }
                __syncwarp();
                if (++st == kPairStages) { st = 0; phase ^= 1; }
            }
            if (!stalled && elect_one()) mma_commit_pair(ready + (n & 1));
            __syncwarp();
        }
        // products in flight end before their tiles and tensor memory go, whichever warp gave up
        if (elect_one()) mma_commit_pair(over);
        __syncwarp();
        if (!warp_drain(over, 0)) stalled = true;
    } else if (warp >= 4) {
        // two warps to a quarter of the lanes, 128 columns each
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        float* staged = reinterpret_cast<float*>(smem + PairSmem::staged) + (warp - 4) * 32 * 33;
        const uint32_t room_bar = cluster_addr(smem_u32(room), 0);
        unsigned n = 0;
        for (int64_t t = first; t < tiles; t += step, ++n) {
            int64_t tm, tn;
            pair_tile(t, tiles_m, tiles_n, &tm, &tn);
            const int64_t r0 = (tm * 2 + rank) * kTile + quarter * 32, c0 = tn * kPairTile + half * kTile;
            uint32_t mask[4];
            load_mask(p, r0 + lane, c0, mask);
            if (!wait_long(ready + (n & 1), (n >> 1) & 1, blocks)) { stalled = true; break; }
            tmem_fence_after();
            const uint32_t d = tmem + (uint32_t(quarter * 32) << 16) + (n & 1 ? kSecond : 0) + half * kTile;
            // The half that shares columns with the other accumulator reads those first: the last
            // chunk of the first accumulator, the first of the second one.  The other half is done with the
            // tile before, which is all that the next product needs of it.
            const bool shares = half == (n & 1 ? 0 : 1);
            auto chunk = [&](int q) { return n & 1 ? q : 3 - q; };
            auto leave = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) cluster_arrive(room_bar);
            };
            if (!shares) leave();
            uint32_t v[2][32];
            tmem_load32(d + chunk(0) * 32, v[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                tmem_wait_load(v[q & 1]);
                if (q == 0 && shares) leave();
                if (q < 3) tmem_load32(d + chunk(q + 1) * 32, v[(q + 1) & 1]);       // on its way during the stores
                const int c = chunk(q) * 32;
                if (c0 + c < p.n) {
                    apply_mask(n & 1 ? mask[q] : mask[3 - q], v[q & 1]);
                    if (p.vec) {
                        if (r0 + lane < p.m) store_row<BF16OUT>(p, r0 + lane, c0 + c, v[q & 1]);
                    } else {
                        store_turned<BF16OUT>(p, r0, c0 + c, v[q & 1], staged);
                    }
                }
            }
        }
    }
    if (stalled && lane < 2) cluster_store(cluster_addr(smem_u32(gave_up), lane), 1u);
    if (stalled && lane == 0) atomicAdd(&g_stalled, 1ull);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();                              // both CTAs are done with each other's barriers and tensor memory
    if (warp == 1 && rank == 1) warp_drain(over, 0);         // the products' arrivals on this CTA's barriers
    if (*gave_up) {                              // as a rule every copy has been multiplied
        // Copies in flight end before the pair does.  A stage counts the bytes of both CTAs, of which one may have
        // issued fewer: those bytes are not expected, or, where rank 0 did already, counted as if they had come.
        if (warp == 0 && rank == 0) {
            const int64_t least = issued[0] < issued[1] ? issued[0] : issued[1], most = issued[0] + issued[1] - least;
            for (int64_t i = least; i < most; ++i) {         // kPairStages at most
                const unsigned bytes = 2 * kTileBytes + (i % blocks % 4 == 0 ? 3 * kScaleBytes : 0);
                if (lane == 0) {
                    if (issued[0] < issued[1]) mbar_arrive_expect_tx(full + i % kPairStages, bytes);
                    else mbar_complete_tx(full + i % kPairStages, bytes);
                }
            }
            __syncwarp();
            for (int64_t i = most < kPairStages ? 0 : most - kPairStages; i < most; ++i)
                warp_drain(full + i % kPairStages, unsigned(i / kPairStages) & 1);
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == 2) tmem_free<2>(tmem, 512);
}

// Tensor maps of the operands.
PFN_cuTensorMapEncodeTiled g_encode = nullptr;
std::once_flag g_encode_flag;

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, const void* v, uint64_t inner, uint64_t outer,
                   uint64_t stride, unsigned box_inner, unsigned box_outer, CUtensorMapSwizzle swizzle) {
    std::call_once(g_encode_flag, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled>(fn);
    });
    if (!g_encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {inner, outer};               // what lies past the matrix reads as 0
    const cuuint64_t strides[1] = {stride};
    const cuuint32_t box[2] = {box_inner, box_outer}, estr[2] = {1, 1};
    return with_context([&] {
        return g_encode(map, type, 2, const_cast<void*>(v), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
}

// The codes of an operand whose tiles have `own` of its uncontracted and 128 of the
// contracted axis: n x k codes, or k x n ones (t).
cudaError_t encode_codes(CUtensorMap* map, const uint8_t* v, int64_t n, int64_t k, int64_t ld, bool t, int own) {
    return t ? encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, v, n, k, ld, kTile, kTile, CU_TENSOR_MAP_SWIZZLE_128B)
             : encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, v, k, n, ld, kTile, own, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale entries as rows of 128 words; `count` of them to a copy.  A copy past the last
// tile of a block group brings the next group's entries, or zeros: scales of rows that do not exist.
cudaError_t encode_scales(CUtensorMap* map, const uint8_t* s, int64_t tiles, int64_t k, int count) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, s, 128, tiles * ((k + 511) / 512), kScaleBytes, 128, count,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
}

cudaError_t launch_pair(MatmulArgs p, const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, cudaStream_t st) {
    CUtensorMap map_a, map_b, map_sa, map_sb;
    cudaError_t e = encode_codes(&map_a, a, p.m, p.k, lda, p.a_t, kTile);
    if (e == cudaSuccess) e = encode_codes(&map_b, b, p.n, p.k, ldb, p.b_t, kTile);
    if (e == cudaSuccess) e = encode_scales(&map_sa, p.sa, p.tiles_m, p.k, 1);
    if (e == cudaSuccess) e = encode_scales(&map_sb, p.sb, p.tiles_n, p.k, 2);
    if (e != cudaSuccess) return e;
    const int64_t es = p.bf16 ? 2 : 4;
    p.vec = aligned(p.out, 32) && p.ldo * es % 32 == 0;
    const int64_t tiles = ((p.m + kPairTile - 1) / kPairTile) * ((p.n + kPairTile - 1) / kPairTile);
    const unsigned grid = unsigned(tiles < kSms / 2 ? 2 * tiles : kSms);
    constexpr unsigned bytes = PairSmem::bytes + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    auto* kernel = p.bf16 ? pair_kernel<true> : pair_kernel<false>;
    e = allow_shared(kernel, bytes);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, grid, kPairThreads, bytes, 2, st, map_a, map_b, map_sa, map_sb, p);
}

template <bool SPLIT>
cudaError_t launch_tiles(MatmulArgs p, const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, int split,
                         cudaStream_t st) {
    // rows of an A tile that a copy brings: no more than there are
    const int box_a = p.a_t || p.m >= kTile ? kTile : int((p.m + 7) / 8 * 8);
    p.a_bytes = box_a * kTile;
    CUtensorMap map_a, map_b;
    cudaError_t e = encode_codes(&map_a, a, p.m, p.k, lda, p.a_t, box_a);
    if (e == cudaSuccess) e = encode_codes(&map_b, b, p.n, p.k, ldb, p.b_t, kTile);
    if (e != cudaSuccess) return e;
    const int64_t es = p.bf16 ? 2 : 4;
    p.vec = SPLIT ? aligned(p.out, 4 * es) && p.ldo % 4 == 0 : aligned(p.out, 32) && p.ldo * es % 32 == 0;
    p.stages = (kStageBytes - 4 * 32 * 33 * 4) / (p.a_bytes + kTileBytes + 2 * kScaleBytes);
    const unsigned bytes = TileSmem(p.stages, p.a_bytes).bytes(p.stages) + 1024;
    auto* kernel = p.bf16 ? tile_kernel<SPLIT, true> : tile_kernel<SPLIT, false>;
    e = allow_shared(kernel, kTileMost);
    if (e != cudaSuccess) return e;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    return launch_early(kernel, SPLIT ? tiles * split : tiles < kSms ? tiles : kSms, kThreads, bytes, split, st, map_a, map_b, p,
                        split);
}

// Which kernel: by the time that each would take, in nanoseconds, from a fit to measured calls with weights
// from memory.  A wave is one tile for each SM (or pair of SMs), a block 128 of the summed axis.
//   pair_kernel:           6300 + 318 a block and wave   (256 x 4096 x 4096: 16.5 us measured, 16.5 fitted;
//                                                          2048 x 4096 x 4096: 28.7, 26.7)
//   tile_kernel, persistent: 4300 + 235 a block and wave (256 x 4096 x 4096: 11.9, 11.8; 512 x 11008 x 4096: 27.7, 26.9)
//   tile_kernel, split s:  the same for blocks / s, and 1300 + 200 s + 22 a row to join the shares (1 x 4096 x 4096, s = 4:
//                          8.7, 8.3, and 11.5 unsplit; 256 x 4096 x 4096, s = 2: 12.6, 12.6).  A split
//                          beyond one CTA to an SM never pays (1 x 4096 x 4096, s = 6: 14.9).
cudaError_t launch(const MatmulArgs& p, const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb, cudaStream_t st) {
    const int64_t blocks = (p.k + kTile - 1) / kTile, tiles = p.tiles_m * p.tiles_n;
    const int64_t pairs = ((p.m + kPairTile - 1) / kPairTile) * ((p.n + kPairTile - 1) / kPairTile);
    const int64_t rows = p.m < kTile ? p.m : kTile;
    const int64_t as_pairs = 6300 + 318 * blocks * ((pairs + kSms / 2 - 1) / (kSms / 2));
    int64_t best = 4300 + 235 * blocks * ((tiles + kSms - 1) / kSms);
    int split = 1;
    for (int s = 2; s <= 8 && tiles * s <= kSms && blocks / s >= 2; ++s) {
        const int64_t ns = 4300 + 235 * ((blocks + s - 1) / s) + 1300 + 200 * s + 22 * rows;
        if (ns < best) {
            best = ns;
            split = s;
        }
    }
    if (as_pairs < best) return launch_pair(p, a, lda, b, ldb, st);
    return split > 1 ? launch_tiles<true>(p, a, lda, b, ldb, split, st) : launch_tiles<false>(p, a, lda, b, ldb, 1, st);
}

}  // namespace

#ifdef TSENOR_GIVE_UP
extern "C" int give_up_products(unsigned polls, unsigned one_in) { return give_up(polls, one_in); }
#endif

cudaError_t stalls(unsigned long long** counter) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(counter), g_stalled);
}

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
    if (((m + kTile - 1) / kTile) * ((n + kTile - 1) / kTile) > most / 8) return TSENOR_ERR_SHAPE;
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
    MatmulArgs p{};
    p.sa = scales_a;
    p.sb = scales_b;
    p.m = m;
    p.n = n;
    p.k = k;
    p.mask = mask;
    p.wpr = (n + 31) / 32;
    p.out = out;
    p.ldo = ldo;
    p.tiles_m = (m + kTile - 1) / kTile;
    p.tiles_n = (n + kTile - 1) / kTile;
    p.a_t = a_t;
    p.b_t = b_t;
    p.bf16 = dtype == TSENOR_BF16;
    const cudaError_t e = launch(p, a, lda, b, ldb, st);
    return e == cudaSuccess ? TSENOR_OK : cuda_fail(e, "tsenor_matmul launch");
}
