// mx_matmul.cu -- products of microscaled matrices on the tensor cores:
//
//   out[m, n] = sum_k A[m, k] B[n, k],  A[m, k] = 2^sa[m, k / 32] a[m, k], B alike
//
// Elements and scales go to the tensor cores as they are stored (mx.cuh): TMA brings
// 128 bytes of k of each row and the tiles of scales that belong to them to shared
// memory, the scales go on to tensor memory, the accumulators are fp32.
//
// Two kernels.  Where there are tiles enough for every pair of SMs, a pair takes tiles
// of 256 x 256; else one CTA takes 128 rows of one operand and up to 128 of the other,
// and a cluster of up to 8 shares k, so that few tokens read a weight with every SM.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <utility>

#include "device_utils.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "tcgen05.cuh"
#include "tma_host.h"

namespace {

namespace tc = ss::tc;
using ss::launch_after;
using ss::wait_before;

constexpr int kRowBytes = 128;               // of k a stage
constexpr int kHalf = 128;                   // rows of an operand that a CTA holds
constexpr int kOperand = kHalf * kRowBytes;  // bytes

// Tiles of scales (128 elements of k) a stage, and their bytes for 128 rows.
__host__ __device__ constexpr int scale_tiles(int format) { return format == SS_MXFP4 ? 2 : 1; }
__host__ __device__ constexpr int scale_bytes(int format) { return scale_tiles(format) * ss::kMxTileBytes; }

// data: rows of bytes; scales: words, a row of them for each 128 rows.
struct Maps {
    CUtensorMap a, b, a_scales, b_scales;
};

// After a wait that ran out: copies in flight land before the CTA goes (its other
// roles' since; its own are two seconds old).
__device__ __forceinline__ void let_copies_land() {
    const uint64_t t0 = tc::global_ns();
    while (tc::global_ns() - t0 < 1000000ull) __nanosleep(20000);
}

// Columns of tensor memory for one tile of scales: A's 4, then B's, 4 for each 128 rows.
template <bool PAIR>
__host__ __device__ constexpr int scale_columns() { return PAIR ? 12 : 8; }

// The products of one stage: its scales' copies to tensor memory, then an instruction
// for each 32 bytes of k.  Two sets of columns take turns from one tile of scales to the
// next, so that a copy need not wait for the products that read the ones before.
template <int FORMAT, bool PAIR>
__device__ __forceinline__ void stage_products(uint32_t d, uint32_t scales, int it, uint32_t a, uint32_t b, uint32_t sa,
                                               uint32_t sb, uint32_t idesc, bool accumulate) {
    constexpr bool FOUR = FORMAT == SS_MXFP4;
    constexpr int T = scale_tiles(FORMAT), per = 4 / T;  // instructions for a tile of scales
    const uint64_t da = tc::operand_desc(a, 16, 1024), db = tc::operand_desc(b, 16, 1024);
    const uint32_t first = scales + (T == 1 && (it & 1) ? scale_columns<PAIR>() : 0);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const uint32_t at = first + t * scale_columns<PAIR>();
        tc::copy_scales<PAIR>(at, tc::scale_desc(sa + t * ss::kMxTileBytes));
#pragma unroll
        for (int r = 0; r < (PAIR ? 2 : 1); ++r)
            tc::copy_scales<PAIR>(at + 4 + 4 * r, tc::scale_desc(sb + (r * T + t) * ss::kMxTileBytes));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t step = (uint64_t)(i * 32 >> 4);
        const uint32_t at = first + i / per * scale_columns<PAIR>();
        tc::mma_scaled<PAIR, FOUR>(d, da + step, db + step, idesc + tc::scale_id(FOUR ? 2 * (i % per) : i), at, at + 4,
                                   accumulate || i > 0);
    }
}

// The first n of four neighbouring elements of out.
__device__ __forceinline__ void store_four(void* out, int64_t at, float4 v, int n, int elem_bytes) {
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (elem_bytes == 2) {
        uint16_t* o = static_cast<uint16_t*>(out) + at;
        if (n >= 4 && (reinterpret_cast<uintptr_t>(o) & 7u) == 0) {
            *reinterpret_cast<uint2*>(o) = make_uint2(ss::pack_bf16x2(f[0], f[1]), ss::pack_bf16x2(f[2], f[3]));
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) o[i] = ss::f32_to_bf16(f[i]);
    } else {
        float* o = static_cast<float*>(out) + at;
        if (n >= 4 && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
            *reinterpret_cast<float4*>(o) = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) o[i] = f[i];
    }
}

__device__ __forceinline__ void store_one(void* out, int64_t at, float v, int elem_bytes) {
    if (elem_bytes == 2)
        static_cast<uint16_t*>(out)[at] = ss::f32_to_bf16(v);
    else
        static_cast<float*>(out)[at] = v;
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles, a pair of CTAs each
// ---------------------------------------------------------------------------

constexpr int kTile = 256;
constexpr int kStages = 5;
constexpr int kEpilogueWarps = 8;  // two for each 32 rows, half of the columns each
constexpr int kColumns = kTile / 2;
constexpr int kPairThreads = 32 * (4 + kEpilogueWarps);
// Two accumulators of 256 columns leave no room in tensor memory for the scales, so the
// second one begins inside the first.  The columns that they share are read first.
constexpr int kShared = 32;
constexpr int kScaleColumns = 2 * kTile - kShared;

__host__ __device__ constexpr int pair_stage(int format) {
    return 2 * kOperand + (3 * scale_bytes(format) + 1023) / 1024 * 1024;
}
constexpr int kTurn = 32 * 128;  // bytes of an epilogue warp: 32 rows of 128
__host__ __device__ constexpr int pair_smem(int format) {
    return kStages * pair_stage(format) + kEpilogueWarps * kTurn + 1024;
}

struct PairArgs {
    int64_t M, N, out_stride;
    int m_tiles, n_tiles, k_blocks;
    void* out;
    int elem_bytes;
    int vector;  // rows of out on 16 bytes
    int expire;  // diagnostics: the first pair gets a wait that nothing ends
};

// 32 columns of this lane's row as bf16 words (or fp32 ones) in its warp's shared memory:
// 16-byte groups of row i at group ^ (i & 7), free of bank conflicts both ways.
__device__ __forceinline__ void turn_half(uint32_t* words, int lane, int h, const uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = ss::pack_bf16x2(__uint_as_float(r[8 * i + 2 * e]), __uint_as_float(r[8 * i + 2 * e + 1]));
        *reinterpret_cast<uint4*>(words + lane * 32 + 4 * ((4 * h + i) ^ (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void turn_full(uint32_t* words, int lane, const uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(words + lane * 32 + 4 * (i ^ (lane & 7))) =
            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
}

// The warp's 32 rows of 128 bytes from its shared memory to out, from (row0, col0) on.
__device__ __forceinline__ void write_turned(const PairArgs& g, const uint32_t* words, int lane, int64_t row0, int64_t col0) {
    const int per = g.elem_bytes == 2 ? 2 : 1;  // columns a word
    const int k = lane & 7, left = (int)min(g.N - col0, (int64_t)(32 * per));
    if (g.vector) {
        const int mine = min(left - 4 * per * k, 4 * per);  // columns of this lane's 16 bytes
        if (mine <= 0) return;
        unsigned char* o = static_cast<unsigned char*>(g.out) +
                           ((row0 + (lane >> 3)) * g.out_stride + col0 + 4 * per * k) * g.elem_bytes;
        const int64_t step = 4 * g.out_stride * g.elem_bytes;
#pragma unroll
        for (int i = 0; i < 8; ++i, o += step) {
            const int q = 4 * i + (lane >> 3);
            if (row0 + q >= g.M) return;
            const uint4 v = *reinterpret_cast<const uint4*>(words + q * 32 + 4 * (k ^ (q & 7)));
            if (mine == 4 * per) {
                *reinterpret_cast<uint4*>(o) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e >= mine) continue;
                    if (per == 2)
                        reinterpret_cast<uint16_t*>(o)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                    else if (e < 4)
                        reinterpret_cast<uint32_t*>(o)[e] = w[e];
                }
            }
        }
    } else {
        for (int q = 0; q < 32 && row0 + q < g.M; ++q) {
            const int64_t at = (row0 + q) * g.out_stride + col0;
            const uint32_t w = words[q * 32 + 4 * ((lane >> 2) ^ (q & 7)) + (lane & 3)];
            if (per == 2) {
                uint16_t* o = static_cast<uint16_t*>(g.out) + at;
                if (2 * lane < left) o[2 * lane] = (uint16_t)w;
                if (2 * lane + 1 < left) o[2 * lane + 1] = (uint16_t)(w >> 16);
            } else if (lane < left) {
                static_cast<uint32_t*>(g.out)[at + lane] = w;
            }
        }
    }
}

// Persistent pairs, each a tile of 256 x 256 at a time, its first CTA the upper 128 rows.
// Warp 0 loads, warp 1 of the first CTA issues the products, warps 4.. read finished
// accumulators while the next tile's products go to the other one.
//
// Bound by the tensor cores: a stage's four instructions take the pair 512 clocks in
// either format, for which each CTA reads 35 KB.  The stages of a tile follow one another
// at that pace, 700 clocks pass between tiles, 2400 before the first stage of a launch and
// 4800 behind the last one; pairs without a tile in the last round are what is lost beside
// that.  8192 x 11008 x 4096 in 4 bits 105 us, 7.0 PFLOP/s, where the clock under that
// load would allow 8.9; 8192 x 5632 x 2048 37 us, 5.1; 2048 x 5632 x 2048 in 8 bits 21 us,
// 2.2 (2.3 rounds of tiles take 3).  What made it: the second accumulator (180 -> 165 us),
// operands in uniform registers (-> 118), accumulators given back without a release (->
// 105).  Each CTA loads the scales of all of B's rows, 1 KB (4 bits) more a stage than its
// half: no load is multicast, because a map may be of any address a caller gives (105 us
// either way, 37 and 21 too).
template <int FORMAT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
mx_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PairArgs g) {
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t bars[2 * kStages + 6];
    __shared__ uint32_t tmem_base;
    constexpr int kStage = pair_stage(FORMAT), kScales = scale_bytes(FORMAT);

    launch_after();
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_ctarank();
    const uint32_t smem = (tc::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16, shared_read = acc_empty + 16;
    const uint32_t never = shared_read + 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(acc_full + 8 * i, 1);
            tc::mbar_init(acc_empty + 8 * i, 2 * kEpilogueWarps);
        }
        tc::mbar_init(shared_read, kEpilogueWarps);
        tc::mbar_init(never, 1);
        tc::mbar_init_fence();
        tc::prefetch_map(&maps.a);
        tc::prefetch_map(&maps.b);
        tc::prefetch_map(&maps.a_scales);
        tc::prefetch_map(&maps.b_scales);
    }
    if (warp == 2) tc::tmem_alloc(tc::smem_addr(&tmem_base), 512);
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    wait_before();

    const int first = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int64_t tiles = (int64_t)g.m_tiles * g.n_tiles;
    bool ok = true;

    if (warp == 0) {
        const uint32_t full0 = tc::map_to_rank(full, 0);
        int it = 0;
        for (int64_t id = first; id < tiles && ok; id += pairs) {
            const int m = (int)(id % g.m_tiles), n = (int)(id / g.m_tiles);
            const int a_row = m * kTile + (int)rank * kHalf, b_row = n * kTile + (int)rank * kHalf;
            for (int k = 0; k < g.k_blocks; ++k, ++it) {
                const int st = it % kStages;
                const uint32_t a = smem + st * kStage, b = a + kOperand, sa = b + kOperand, sb = sa + kScales;
                ok = tc::mbar_wait_warp(empty + 8 * st, ((it / kStages) & 1) ^ 1);
                if (!ok) break;
                if (!tc::elect_one()) continue;
                const uint32_t bar = full0 + 8 * st;
                if (rank == 0) tc::mbar_expect_tx(full + 8 * st, 2 * (2 * kOperand + 3 * kScales));
                tc::tma_load_2d(a, &maps.a, k * kRowBytes, a_row, bar);
                tc::tma_load_2d(sa, &maps.a_scales, k * (kScales / 4), m * 2 + (int)rank, bar);
                tc::tma_load_2d(b, &maps.b, k * kRowBytes, b_row, bar);
                // the scales of all of B's rows, two rows of tiles: each CTA multiplies with both
                tc::tma_load_2d(sb, &maps.b_scales, k * (kScales / 4), n * 2, bar);
            }
        }
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = tc::scaled_desc(FORMAT == SS_MXFP4, kTile, kTile);
        int it = 0, j = 0;
        if (g.expire && first == 0) ok = tc::mbar_wait_warp(never, 0);
        for (int64_t id = first; id < tiles && ok; id += pairs, ++j) {
            ok = tc::mbar_wait_warp(acc_empty + 8 * (j & 1), ((j >> 1) & 1) ^ 1) &&
                 (j == 0 || tc::mbar_wait_warp(shared_read, (j - 1) & 1));
            if (!ok) break;
            tc::fence_after();
            const uint32_t d = tmem + (j & 1) * (kTile - kShared);
            for (int k = 0; k < g.k_blocks; ++k, ++it) {
                const int st = it % kStages;
                const uint32_t a = smem + st * kStage, b = a + kOperand, sa = b + kOperand, sb = sa + kScales;
                ok = tc::mbar_wait_warp(full + 8 * st, (it / kStages) & 1);
                if (!ok) break;
                tc::fence_after();
                if (tc::elect_one()) {
                    stage_products<FORMAT, true>(d, tmem + kScaleColumns, it, a, b, sa, sb, idesc, k > 0);
                    tc::commit_pair(empty + 8 * st);
                    if (k + 1 == g.k_blocks) tc::commit_pair(acc_full + 8 * (j & 1));
                }
                __syncwarp();
            }
            if (!ok) break;
        }
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t acc_empty0 = tc::map_to_rank(acc_empty, 0), shared_read0 = tc::map_to_rank(shared_read, 0);
        uint32_t* words = reinterpret_cast<uint32_t*>(raw + (smem - tc::smem_addr(raw)) + kStages * kStage +
                                                      (warp - 4) * kTurn);
        const int wide = g.elem_bytes == 2 ? 64 : 32, pieces = kColumns / wide;  // columns a piece
        int j = 0;
        for (int64_t id = first; id < tiles; id += pairs, ++j) {
            const int m = (int)(id % g.m_tiles), n = (int)(id / g.m_tiles);
            const int64_t row0 = (int64_t)m * kTile + rank * kHalf + quad * 32;
            const int64_t col0 = (int64_t)n * kTile + half * kColumns;
            const uint32_t d = tmem + (j & 1) * (kTile - kShared) + half * kColumns + ((uint32_t)quad << 21);
            // the shared columns are the first accumulator's last and the second one's first
            const bool shares = half != (j & 1);
            const int start = shares && half ? pieces - 1 : 0;
            ok = ok && tc::mbar_wait(acc_full + 8 * (j & 1), (j >> 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc::fence_after();
#pragma unroll 1
            for (int i = 0; i < pieces; ++i) {
                const int c = (start + i) % pieces * wide;
                uint32_t r[2][32];
                __syncwarp();
                tc::tmem_ld32(d + c, r[0]);
                if (wide == 64) tc::tmem_ld32(d + c + 32, r[1]);
                tc::tmem_wait(r[0]);
                if (wide == 64) tc::tmem_wait(r[1]);
                tc::fence_before();
                __syncwarp();
                if (lane == 0 && i == 0 && shares) tc::mbar_arrive_read(shared_read0);
                if (lane == 0 && i + 1 == pieces) tc::mbar_arrive_read(acc_empty0 + 8 * (j & 1));
                if (!ok) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[0][e] = r[1][e] = 0x7FFFFFFFu;
                }
                if (row0 >= g.M || col0 + c >= g.N) continue;
                if (wide == 64) {
                    turn_half(words, lane, 0, r[0]);
                    turn_half(words, lane, 1, r[1]);
                } else {
                    turn_full(words, lane, r[0]);
                }
                __syncwarp();
                write_turned(g, words, lane, row0, col0 + c);
            }
        }
    }
    if (!ok) let_copies_land();
    __syncwarp();
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    if (warp == 2) tc::tmem_free(tmem, 512);
}

// ---------------------------------------------------------------------------
// 128 rows of one operand, few of the other, k over a cluster
// ---------------------------------------------------------------------------

constexpr int kFewStages = 4;
constexpr int kFewThreads = 32 * 8;  // loader, issuer, four that read the accumulator; all join the shares

__host__ __device__ constexpr int few_stage(int format, int few) {
    return kOperand + few * kRowBytes + 2 * scale_bytes(format);
}
__host__ __device__ constexpr int few_smem(int format, int few) { return kFewStages * few_stage(format, few) + 1024; }
// Columns of tensor memory: the accumulator's and the scales' 16.
__host__ __device__ constexpr uint32_t few_tmem(int few) { return few <= 16 ? 32 : 2 * few; }

// Few rows are bound by the weight's read, and by the chain of a launch: 1800 clocks until
// the first stage is there, 500 a stage from then on, 1500 for the sums to be in shared
// memory and 1500 for the join.  One token through 11008 x 4096 in 4 bits (24 MB): 5.5 us
// behind the launch that quantises it; 1021 x 777 x 1001: 5.6 us.
//
// a: the operand of 128 rows a CTA; b: the other one.
struct FewArgs {
    int64_t rows, few;           // of the two operands
    int64_t row_step, few_step;  // elements of out between two rows of a, of b
    int row_tiles, k_blocks, splits;
    void* out;
    int elem_bytes;
    int vector;  // out's four neighbouring elements lie on their size
    int expire;  // diagnostics: the first CTA gets a wait that nothing ends
};

template <int FORMAT, int FEW>
__global__ void __launch_bounds__(kFewThreads) mx_few_kernel(const __grid_constant__ Maps maps,
                                                            const __grid_constant__ FewArgs g) {
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t bars[2 * kFewStages + 2];
    __shared__ uint32_t tmem_base;
    constexpr int kStage = few_stage(FORMAT, FEW), kScales = scale_bytes(FORMAT);
    static_assert(kStage % 1024 == 0 && (FEW + 8 * kFewThreads / 32) * kHalf * 4 <= kFewStages * kStage, "shared memory");

    launch_after();
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t smem = (tc::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kFewStages, done = empty + 8 * kFewStages;
    const uint32_t never = done + 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kFewStages; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        tc::mbar_init(done, 1);
        tc::mbar_init(never, 1);
        tc::mbar_init_fence();
        tc::prefetch_map(&maps.a);
        tc::prefetch_map(&maps.b);
        tc::prefetch_map(&maps.a_scales);
        tc::prefetch_map(&maps.b_scales);
    }
    if (warp == 1) tc::tmem_alloc_one(tc::smem_addr(&tmem_base), few_tmem(FEW));
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    wait_before();

    float* part_all = reinterpret_cast<float*>(raw + (smem - tc::smem_addr(raw)));
    const int split = g.splits > 1 ? (int)tc::cluster_ctarank() : 0;
    const int tile = blockIdx.x / g.splits, rt = tile % g.row_tiles, ft = tile / g.row_tiles;
    const int per = (g.k_blocks + g.splits - 1) / g.splits;
    const int kb = min(split * per, g.k_blocks), ke = min(kb + per, g.k_blocks);
    bool ok = true;

    if (warp == 0) {
        for (int k = kb; k < ke; ++k) {
            const int it = k - kb, st = it % kFewStages;
            const uint32_t a = smem + st * kStage, b = a + kOperand, sa = b + FEW * kRowBytes, sb = sa + kScales;
            ok = tc::mbar_wait_warp(empty + 8 * st, ((it / kFewStages) & 1) ^ 1);
            if (!ok) break;
            if (!tc::elect_one()) continue;
            tc::mbar_expect_tx(full + 8 * st, kOperand + FEW * kRowBytes + 2 * kScales);
            tc::tma_load_2d_one(a, &maps.a, k * kRowBytes, rt * kHalf, full + 8 * st);
            tc::tma_load_2d_one(sa, &maps.a_scales, k * (kScales / 4), rt, full + 8 * st);
            tc::tma_load_2d_one(b, &maps.b, k * kRowBytes, ft * FEW, full + 8 * st);
            tc::tma_load_2d_one(sb, &maps.b_scales, k * (kScales / 4), ft, full + 8 * st);
        }
    } else if (warp == 1) {
        const uint32_t idesc = tc::scaled_desc(FORMAT == SS_MXFP4, kHalf, FEW);
        if (g.expire && blockIdx.x == 0) ok = tc::mbar_wait_warp(never, 0);
        for (int k = kb; k < ke && ok; ++k) {
            const int it = k - kb, st = it % kFewStages;
            const uint32_t a = smem + st * kStage, b = a + kOperand, sa = b + FEW * kRowBytes, sb = sa + kScales;
            ok = tc::mbar_wait_warp(full + 8 * st, (it / kFewStages) & 1);
            if (!ok) break;
            tc::fence_after();
            if (tc::elect_one()) {
                stage_products<FORMAT, false>(tmem, tmem + FEW, it, a, b, sa, sb, idesc, k > kb);
                tc::commit_one(empty + 8 * st);
                if (k + 1 == ke) tc::commit_one(done);
            }
            __syncwarp();
        }
        if (kb == ke && tc::elect_one()) tc::commit_one(done);
    } else if (warp >= 2 && warp < 6) {
        const int quad = warp & 3, row = quad * 32 + lane;
        ok = tc::mbar_wait(done, 0);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc::fence_after();
        // every stage has been read: its shared memory takes the sums
        float* part = part_all;
        const bool none = kb == ke;  // no k: the accumulator holds something else
#pragma unroll 1
        for (int c = 0; c < FEW; c += 32) {
            uint32_t r[32];
            __syncwarp();
            tc::tmem_ld32(tmem + c + ((uint32_t)quad << 21), r);
            tc::tmem_wait(r);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i < FEW) part[(c + i) * kHalf + row] = !ok ? NAN : none ? 0.f : __uint_as_float(r[i]);
        }
    }
    if (!ok) let_copies_land();
    __syncwarp();
    tc::fence_before();
    if (g.splits > 1)
        tc::cluster_sync();
    else
        __syncthreads();
    tc::fence_after();
    if (warp == 1) tc::tmem_free_one(tmem, few_tmem(FEW));

    // this CTA's share of the columns, the splits added in their order; eight columns a warp at a
    // time, so that as many loads from the other CTAs are on their way
    const int share = (FEW + g.splits - 1) / g.splits, c0 = split * share;
    const int64_t few0 = (int64_t)ft * FEW;
    const int columns = (int)min(min((int64_t)c0 + share, (int64_t)FEW), g.few - few0) - c0;  // that exist
    if (g.row_step == 1) {
        const int64_t r = (int64_t)rt * kHalf + 4 * lane;
        const int have = (int)min(g.rows - r, (int64_t)4);
        for (int c = 8 * warp; c < columns; c += 8 * (kFewThreads / 32)) {
            float4 s[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) s[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int q = 0; q < g.splits; ++q) {
                const uint32_t at = tc::map_to_rank(smem + (uint32_t)((c0 + c) * kHalf + 4 * lane) * 4, q);
                float4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (c + u < columns)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v[u].x), "=f"(v[u].y), "=f"(v[u].z), "=f"(v[u].w)
                                     : "r"(at + u * kHalf * 4));
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (c + u < columns) s[u].x += v[u].x, s[u].y += v[u].y, s[u].z += v[u].z, s[u].w += v[u].w;
            }
            if (g.vector) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (c + u < columns) store_four(g.out, r + (few0 + c0 + c + u) * g.few_step, s[u], have, g.elem_bytes);
            } else {  // lanes along the row, through the shared memory behind the sums
                float* mine = part_all + FEW * kHalf + warp * 8 * kHalf;
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u) *reinterpret_cast<float4*>(mine + u * kHalf + 4 * lane) = s[u];
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int64_t at = (int64_t)rt * kHalf + (few0 + c0 + c + u) * g.few_step;
#pragma unroll
                    for (int k = lane; k < kHalf; k += 32)
                        if (c + u < columns && (int64_t)rt * kHalf + k < g.rows)
                            store_one(g.out, at + k, mine[u * kHalf + k], g.elem_bytes);
                }
            }
        }
    } else {  // out is contiguous along the few: a row a lane, four columns at a time
        const int row = threadIdx.x & (kHalf - 1);
        const int64_t r = (int64_t)rt * kHalf + row;
        for (int c = 4 * (threadIdx.x / kHalf); c < columns && r < g.rows; c += 4 * (kFewThreads / kHalf)) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < g.splits; ++q) {
                const uint32_t at = tc::map_to_rank(smem + (uint32_t)((c0 + c) * kHalf + row) * 4, q);
                float v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[u]) : "r"(at + u * kHalf * 4));
#pragma unroll
                for (int u = 0; u < 4; ++u) s[u] += v[u];
            }
            store_four(g.out, r * g.row_step + few0 + c0 + c, make_float4(s[0], s[1], s[2], s[3]), min(columns - c, 4),
                       g.elem_bytes);
        }
    }
    __syncwarp();
    if (g.splits > 1) tc::cluster_sync_read();
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

constexpr int64_t kMaxSize = (int64_t)1 << 30;

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Data of a quantised matrix in boxes of 128 bytes and box_rows rows, zeros outside.
int data_map(CUtensorMap* map, const void* data, int64_t rows, int64_t K, int format, int box_rows) {
    const ss::EncodeTiled fn = ss::tensor_map_encoder();
    if (!fn) return ss::cuda_fail(cudaErrorNotSupported);
    const cuuint64_t pitch = (cuuint64_t)div_up(K, ss::kMxTile) * (format == SS_MXFP4 ? 64 : 128);
    const cuuint64_t dims[2] = {pitch, (cuuint64_t)rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {kRowBytes, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(data), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SS_OK : ss::cuda_fail(cudaErrorInvalidValue);
}

// Its scales, as words, in boxes of a stage's tiles for box_tiles times 128 rows; zeros,
// which are the lowest scale, outside.
int scale_map(CUtensorMap* map, const void* scales, int64_t rows, int64_t K, int format, int box_tiles) {
    const ss::EncodeTiled fn = ss::tensor_map_encoder();
    if (!fn) return ss::cuda_fail(cudaErrorNotSupported);
    const cuuint64_t pitch = (cuuint64_t)div_up(K, ss::kMxTile) * ss::kMxTileBytes;
    const cuuint64_t dims[2] = {pitch / 4, (cuuint64_t)div_up(rows, ss::kMxTile)}, strides[1] = {pitch};
    const cuuint32_t box[2] = {(cuuint32_t)scale_bytes(format) / 4, (cuuint32_t)box_tiles}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<void*>(scales), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SS_OK : ss::cuda_fail(cudaErrorInvalidValue);
}

struct Operand {
    const void *data, *scales;
    int64_t rows;
};

// b_rows: of a box of B; b_tiles: rows of tiles in one of its scales.
int make_maps(Maps* maps, const Operand& a, const Operand& b, int64_t K, int format, int b_rows, int b_tiles) {
    if (int rc = data_map(&maps->a, a.data, a.rows, K, format, kHalf)) return rc;
    if (int rc = data_map(&maps->b, b.data, b.rows, K, format, b_rows)) return rc;
    if (int rc = scale_map(&maps->a_scales, a.scales, a.rows, K, format, 1)) return rc;
    return scale_map(&maps->b_scales, b.scales, b.rows, K, format, b_tiles);
}

template <int FORMAT>
int launch_pair(const ss_mx_product* p, int64_t k_blocks, bool expire, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const auto kernel = mx_pair_kernel<FORMAT>;
    constexpr int smem = pair_smem(FORMAT);
    if (int rc = ss::allow_smem(ready, reinterpret_cast<const void*>(kernel), smem)) return rc;
    Maps maps;
    if (int rc = make_maps(&maps, {p->a_data, p->a_scales, p->M}, {p->b_data, p->b_scales, p->N}, p->K, FORMAT, kHalf, 2))
        return rc;
    const int64_t m_tiles = div_up(p->M, kTile), n_tiles = div_up(p->N, kTile), pairs = ss::num_sms() / 2;
    const PairArgs g = {p->M, p->N, p->out_stride, (int)m_tiles, (int)n_tiles, (int)k_blocks, p->out, p->elem_bytes,
                        ss::aligned(p->out, 16) && p->out_stride * p->elem_bytes % 16 == 0, expire};
    return ss::launch(kernel, 2 * std::min(m_tiles * n_tiles, pairs), kPairThreads, smem, 0, true, st, maps, g);
}

// CTAs that share k: as many as make the time least, counted in k blocks of a CTA (0.19
// us), of which a second CTA on an SM costs 0.7, and a share's join as much as a
// forty-fifth of a block for each column.  All of them are held at once; clusters of 7
// and 8 waste SMs of a GPC and are taken where that does not matter.  One token, 2048 x
// 2048: 4.0 us alone, 3.6 with 4, 4.3 with 8; 11008 x 4096: 6.3 alone, 5.6 with 3, 8.7
// with 4; 128 tokens, 2048 x 2048: 6.2 alone, 5.6 with 2, 7.1 with 4, 17 with 8.
int choose_splits(int64_t tiles, int64_t k_blocks, int few, int smem) {
    const int64_t sms = ss::num_sms(), each = smem <= 112 * 1024 ? 2 : 1;  // CTAs an SM holds
    int best = 1;
    double least = INFINITY;
    for (int s = 1; s <= 8 && s <= k_blocks; ++s) {
        if (s > 1 && tiles * s * (s > 6 ? 2 : 1) > sms * each) continue;
        const int64_t n = div_up(tiles * s, sms);
        const double load = (double)(n / each) * (each == 2 ? 1.7 : 1.0) + (double)(n % each);
        const double cost = load * (double)div_up(k_blocks, s) + (s - 1) * few / 45.0;
        if (cost < least) best = s, least = cost;
    }
    return best;
}

template <int FORMAT, int FEW>
int launch_few(const ss_mx_product* p, int64_t k_blocks, bool swap, bool expire, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const auto kernel = mx_few_kernel<FORMAT, FEW>;
    constexpr int smem = few_smem(FORMAT, FEW);
    if (int rc = ss::allow_smem(ready, reinterpret_cast<const void*>(kernel), smem)) return rc;
    Operand a = {p->b_data, p->b_scales, p->N}, b = {p->a_data, p->a_scales, p->M};
    if (swap) std::swap(a, b);
    Maps maps;
    if (int rc = make_maps(&maps, a, b, p->K, FORMAT, FEW, 1)) return rc;
    const int64_t row_tiles = div_up(a.rows, kHalf), few_tiles = div_up(b.rows, FEW), tiles = row_tiles * few_tiles;
    const int splits = choose_splits(tiles, k_blocks, FEW, smem);
    const FewArgs g = {a.rows, b.rows, swap ? p->out_stride : 1, swap ? 1 : p->out_stride, (int)row_tiles, (int)k_blocks,
                       splits, p->out, p->elem_bytes,
                       ss::aligned(p->out, 4 * p->elem_bytes) && p->out_stride % 4 == 0, expire};
    if (tiles * splits > INT32_MAX) return SS_EOVERFLOW;
    return ss::launch(kernel, tiles * splits, kFewThreads, smem, splits > 1 ? splits : 0, true, st, maps, g);
}

// The next call gets a wait which nothing ends.
std::atomic<bool> g_expire{false};

template <int FORMAT>
int launch_product(const ss_mx_product* p, cudaStream_t st) {
    const bool expire = g_expire.exchange(false, std::memory_order_relaxed);
    const int64_t k_blocks = div_up(div_up(p->K, ss::kMxTile), scale_tiles(FORMAT));
    const int64_t big = div_up(p->M, kTile) * div_up(p->N, kTile);
    // half a round of tiles: 36 of them take the same either way (1536 x 1536 x 4096: 8.4 and 8.6 us),
    // 16 are faster as the few (1021 x 777 x 4096: 7.0 and 10.1), 44 as pairs (512 x 5632 x 4096: 16 and 9.2)
    if (2 * big >= ss::num_sms() / 2 && p->M > kHalf && p->N > kHalf) return launch_pair<FORMAT>(p, k_blocks, expire, st);
    // the few are A's rows, or B's where those are no more than a tile (5003 x 72 x 2688: 7.4 us as A's,
    // 6.8 as B's; 2000 x 100 x 4096 in 8 bits 9.0 and 6.6, in 4 bits 7.0 and 7.3); with more of them a row
    // of out in one thread's hands costs more (1021 x 777 x 1024: 5.7 and 17)
    const bool swap = p->N < p->M && p->N <= kHalf;
    const int64_t few = swap ? p->N : p->M;
    if (few <= 16) return launch_few<FORMAT, 16>(p, k_blocks, swap, expire, st);
    if (few <= 32) return launch_few<FORMAT, 32>(p, k_blocks, swap, expire, st);
    if (few <= 64) return launch_few<FORMAT, 64>(p, k_blocks, swap, expire, st);
    return launch_few<FORMAT, 128>(p, k_blocks, swap, expire, st);
}

}  // namespace

extern "C" int ss_mx_expire_wait(int on) {
    if (on != 0 && on != 1) return SS_EINVAL;
    g_expire.store(on != 0, std::memory_order_relaxed);
    return SS_OK;
}

extern "C" int ss_mx_matmul(const ss_mx_product* p, ss_stream_t stream) {
    if (!p || p->M < 0 || p->N < 0 || p->K < 1 || (p->format != SS_MXFP4 && p->format != SS_MXFP8) ||
        (p->elem_bytes != 2 && p->elem_bytes != 4))
        return SS_EINVAL;
    if (p->M > kMaxSize || p->N > kMaxSize || p->K > kMaxSize) return SS_EOVERFLOW;
    if (p->M == 0 || p->N == 0) return SS_OK;
    if (!p->a_data || !p->a_scales || !p->b_data || !p->b_scales || !p->out || p->out_stride < p->N) return SS_EINVAL;
    if (p->out_stride > INT64_MAX / 8 / p->M) return SS_EOVERFLOW;
    if (!ss::aligned(p->a_data, 16) || !ss::aligned(p->a_scales, 16) || !ss::aligned(p->b_data, 16) ||
        !ss::aligned(p->b_scales, 16) || !ss::aligned(p->out, (uintptr_t)p->elem_bytes))
        return SS_EALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return p->format == SS_MXFP4 ? launch_product<SS_MXFP4>(p, st) : launch_product<SS_MXFP8>(p, st);
}
