// linear_ce.cu -- softmax cross entropy of a linear head over a large
// vocabulary, and its gradients, without keeping the logits.
//
//   l_tv = <h_t, w_v>          lse_t = log sum_v exp(l_tv)
//   loss_t = lse_t - l_t,y(t)  over the tokens whose target is not ignored
//   P_tv = exp(l_tv - lse_t) - [v = y(t)]
//   dH = scale * P W           dW = scale * P^T H
//
// The tokens that count are gathered first, so that ignored ones cost nothing
// and whatever their rows hold (NaN, infinities) stays out of every product.
// Then four matrix products carry the work, 2TVD flops each:
//
//   statistics  H W^T a tile at a time; of each tile's row only the maximum's
//               exponent and the sum of exponentials leave the SM
//   for each piece of the vocabulary (as much of P as the workspace holds):
//     probability  H W^T again, P written in bf16
//     head         dW of the piece = P^T H
//     hidden       dH += P W of the piece
//
// P in bf16 is the one rounding between inputs and outputs beside their own:
// the tensor cores take bf16 operands, and the error it leaves (at most 2^-8 of
// each term, independent) is the size of the outputs' own rounding.  Logits,
// statistics and every sum are fp32, statistics with whole exponents so that
// joining tiles rounds only sums; the tokens' losses are summed in fp64.
//
// Forming the logits twice makes it 8TVD flops for 6TVD, and nothing of size TV is
// kept beyond a piece (which holds all of P up to 4096 tokens at vocabulary 32000).
// 8192 tokens, 32000 x 2048, with gradients: 2640 to 2710 us back to back by the
// device, 1590 to 1630 TFLOP/s of the 8TVD, where a bare library product of such sizes
// sustains 1724 under the card's power limit; 4096 tokens scored at hidden size
// 4096: 630 to 650 us, 1650 to 1700 TFLOP/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "device_utils.cuh"
#include "internal.h"
#include "launch.cuh"
#include "segmap.cuh"
#include "tcgen05.cuh"

namespace {

namespace tc = ss::tc;

constexpr int kTile = 256;        // rows and columns of a CTA pair's tile
constexpr int kHalf = 128;        // each CTA's rows of A, of B, and of the accumulator
constexpr int kBlockK = 64;       // k of one stage: 128 bytes of bf16
constexpr int kStages = 6;
constexpr int kStageBytes = 2 * kHalf * kBlockK * 2;  // A and B of one CTA
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kEpilogueWarps = 8;      // two for each 32 rows, half of the columns each
constexpr int kColumns = kTile / 2;    // of a warp
constexpr int kGemmThreads = 32 * (4 + kEpilogueWarps);

constexpr double kLog2eDouble = 1.4426950408889634;
constexpr float kLog2e = (float)kLog2eDouble;
// The tensor cores' accumulator drops what an add shifts out, towards zero, so a
// logit comes out smaller by a part of itself that grows with the adds: half a unit
// of the running sum's last place for each 16 products behind the ones that made it.
// How large the part is depends on where along k a logit comes from.  Measured
// against 64 bits, for each 16 products: 1.47e-8 to 1.64e-8 for random inputs (hidden
// sizes 256 to 16384, logits of scale 0.3 to 7.7); with one dominant channel and noise,
// 2.7e-8 to 4.1e-8 where the channel comes first, 1.3e-8 to 2.2e-8 in the middle,
// nothing where it comes last; logits that grow evenly along k 1.3e-8 at 1024 and 3.5e-8
// at 4096; products all of one sign that are tiny beside the sum, 1.9e-7.
// The logits' exponent makes good a part near the middle of these, which leaves an
// error of either sign where there was one of one sign; it holds for none of them
// exactly, and is not raised beyond the hidden sizes that it was measured at.
// Loss of 4096 random tokens at hidden size 4096, relative error against 64 bits:
// 1.1e-6 without, 6e-8 with it (fp32 products: 5.9e-7 to 6.5e-7).
constexpr double kDropped = 1.55e-8;
constexpr int64_t kDroppedUpTo = 16384;

constexpr float kLn2High = 0.693145751953125f;                               // 16 bits
constexpr float kLn2Low = (float)(0.6931471805599453 - 0.693145751953125);

// What the gather leaves for the kernels after it, at the workspace's start.
struct Header {
    int live;      // tokens that count
    float scale;   // of both gradients
    int finished;  // CTAs of the loss kernel that are done
    int failed;    // a wait of this call has run out: nothing behind it means anything
};

// The products, by what is done with a 256 x 256 tile of them.
enum Product { kStatistics, kProbability, kHead, kHidden };

// One product of a launch.
struct Work {
    int product;
    int n_tiles;  // column tiles
    int m_tiles;  // row tiles (kHead; the others have token rows: header->live)
    int splits;   // of k (kHead, kHidden)
    int k;        // elements of k (kHead: the tokens that count)
    int v0;       // first vocabulary row of the piece
    // kHead, kHidden: into fp32 partials [splits][rows][part_ld], or, where NULL, into out
    float* part;
    int64_t part_split;  // elements between two splits
    int part_ld;
    int add;             // partials already hold the earlier pieces
    uint16_t* out;
    int64_t out_ld;
    int m_rows;          // rows that exist (kHead)
    int cols;            // columns that exist
    uint16_t* p;         // kProbability: [rows][ldp]
    int ldp;
};

constexpr int kMaxWork = 3;

struct GemmArgs {
    Header* header;
    int* next;  // tiles handed out beyond the first of each pair, 0 at the launch
    int vocab;
    int rows;   // allocated token rows
    float log2e;  // of logits as the products leave them (kDropped)
    float* loss;
    const double* partials;  // this launch sums them to the loss (NULL: it does not)
    int n_partials;
    int mean;
    int expire;              // diagnostics: put in a wait that nothing ends
    const int* target;       // [rows]
    const int* token;        // [rows]: output row of each row (kHidden)
    const float2* row_loss;  // [rows]: log-sum-exp in base 2, the target's p - 1 (kProbability)
    float2* stats;           // [2 n_tiles][rows], each half tile's: exponent of the maximum, sum of exponentials (kStatistics)
    int count;               // products, the ones with the longest tiles first
    Work work[kMaxWork];
};

// The operands of each product.
struct Maps {
    CUtensorMap a[kMaxWork], b[kMaxWork];
};

using ss::launch_after;
using ss::wait_before;

// 2^x: one instruction, good to 2 ulp, results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// This thread's row: exponentials of 32 logits (columns from col of the tile's
// row) added to (m, s), m an integer exponent at or above every logit so far.  The
// maximum passes over NaN, the sum does not: what it holds is never dropped.
__device__ __forceinline__ void add_logits(const uint32_t (&r)[32], float log2e, float& m, float& s) {
    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = __uint_as_float(r[i]);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = fmaxf(top, l[i]);
    const float up = fmaxf(m, ceilf(top * log2e));
    // nothing but -inf so far: any finite exponent gives the zeros it should
    const float at = up == -INFINITY ? 0.f : up;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        a += ex2(fmaf(l[i], log2e, -at));
        b += ex2(fmaf(l[i + 1], log2e, -at));
    }
    s = (m == -INFINITY ? s : s * ex2(m - at)) + (a + b);  // at -inf s is 0, or the NaN of a logit
    m = up;
}

// A wait has run out: every loss from here on is NaN.  The flag first, then the loss,
// as the launch may be summing it at this moment: whichever of the two fences (the other
// is behind that store) comes first, the last store is a NaN.
__device__ __forceinline__ void give_up(Header* header, float* loss) {
    *static_cast<volatile int*>(&header->failed) = 1;
    __threadfence();
    *static_cast<volatile float*>(loss) = NAN;
}

// The loss, by one warp: the partials' sum in a fixed order, over the tokens that
// count for a mean, 0 when there are none.
__device__ __forceinline__ void sum_losses(const double* partials, int n, int live, int mean, float* loss) {
    const int lane = threadIdx.x & 31;
    double s = 0.0;
#pragma unroll 8
    for (int i = lane; i < n; i += 32) s += __ldcg(partials + i);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_down_sync(0xFFFFFFFFu, s, k);
    if (lane == 0) *static_cast<volatile float*>(loss) = (float)(mean && live > 0 ? s / live : s);
}

// This lane's row, columns 32 h .. of 64, as bf16 words in its warp's shared memory.
__device__ __forceinline__ void turn_words(uint32_t* words, int lane, int h, const uint32_t (&r)[32], float scale,
                                           bool none) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = none ? 0u
                        : ss::pack_bf16x2(scale * __uint_as_float(r[8 * i + 2 * e]),
                                          scale * __uint_as_float(r[8 * i + 2 * e + 1]));
        *reinterpret_cast<uint4*>(words + lane * 32 + 4 * ((4 * h + i) ^ (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A tile of a launch: which product (-1: there is none left), where, and its
// split's k blocks.
struct __align__(16) Tile {
    int w, m, n, s, kb, ke, pad[2];
};

// Tiles are numbered product after product.  Token products run down the tokens
// first: the hidden states stay in L2 and the weight is read once.  The gradients
// run along the hidden size first: a panel of P is read by the pairs that need it
// at about the same time.
__device__ __forceinline__ Tile find_tile(const GemmArgs& g, int live, int id) {
    Tile t = {};
    for (int w = 0; w < g.count; ++w) {
        const Work& x = g.work[w];
        const int m_tiles = x.product == kHead ? x.m_tiles : (live + kTile - 1) / kTile;
        const int mn = m_tiles * x.n_tiles, tiles = mn * x.splits;
        if (id >= tiles) {
            id -= tiles;
            continue;
        }
        const int kblocks = ((x.product == kHead ? live : x.k) + kBlockK - 1) / kBlockK;
        const int per = (kblocks + x.splits - 1) / x.splits;
        t.w = w;
        t.s = id / mn;
        id -= t.s * mn;
        if (x.product <= kProbability)
            t.m = id % m_tiles, t.n = id / m_tiles;
        else
            t.m = id / x.n_tiles, t.n = id % x.n_tiles;
        t.kb = min(t.s * per, kblocks);
        t.ke = min(t.kb + per, kblocks);
        return t;
    }
    t.w = -1;
    return t;
}

__device__ __forceinline__ int total_tiles(const GemmArgs& g, int live) {
    int n = 0;
    for (int w = 0; w < g.count; ++w) {
        const Work& x = g.work[w];
        n += (x.product == kHead ? x.m_tiles : (live + kTile - 1) / kTile) * x.n_tiles * x.splits;
    }
    return n;
}

constexpr int kQueue = 4;   // tiles handed out ahead

// One persistent CTA pair takes output tiles of 256 x 256, its first CTA the
// upper 128 rows.  Warp 0 loads (one thread), warp 1 of the first CTA issues the
// products, warps 4.. read finished accumulators from tensor memory while the
// next tile's products go to the other half of it.  Warp 3 of the first CTA hands
// out tiles: a pair's first by its number, then whichever is next of the launch, so
// that products with tiles of different lengths share a launch and the pairs end
// together.  A tile's result does not depend on who computes it.
//
// Bound by the tensor cores: a k block of a tile takes the pair 512 clocks, for
// which each CTA reads 32 KB, 64 bytes a clock, from L2; half the tile would need
// half as much again.  Two accumulators fill tensor memory, and 6 stages what shared
// memory the epilogues' turning leaves.  Tensor pipe active, by launch, at 2048
// tokens, 32000 x 2048: statistics 75 % (156 us, 14 rounds of tiles for 13.2),
// probabilities 72 % (165 us, and 131 MB written), both gradients 85 % (281 us).
// With 4 epilogue warps products of 16 k blocks waited for them (1021 ragged tokens
// 274 -> 238 us with 8); a launch for each product left 7 to 16 % of the last rounds
// empty.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
ce_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ GemmArgs g) {
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) float turn[kEpilogueWarps][32 * 32];
    __shared__ uint64_t bars[2 * kStages + 4 + 2 * kQueue + 1];
    __shared__ Tile queue[kQueue];
    __shared__ uint32_t tmem_base;

    launch_after();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_ctarank();
    const uint32_t smem = (tc::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kStages;
    const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16;
    const uint32_t queue_full = acc_empty + 16, queue_empty = queue_full + 8 * kQueue;
    const uint32_t never = queue_empty + 8 * kQueue;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full + 8 * i, 1);
            tc::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(acc_full + 8 * i, 1);
            tc::mbar_init(acc_empty + 8 * i, 2 * kEpilogueWarps);
        }
        for (int i = 0; i < kQueue; ++i) {
            tc::mbar_init(queue_full + 8 * i, 1);
            tc::mbar_init(queue_empty + 8 * i, 2 + 1 + 2 * kEpilogueWarps);  // loaders, issuer, epilogues
        }
        tc::mbar_init(never, 1);
        tc::mbar_init_fence();
        for (int w = 0; w < g.count; ++w) {
            tc::prefetch_map(&maps.a[w]);
            tc::prefetch_map(&maps.b[w]);
        }
    }
    if (warp == 2) tc::tmem_alloc(tc::smem_addr(&tmem_base), 512);
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    wait_before();

    const int live = g.header->live;
    const int first = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    bool ok = true;

    // The pair's j-th tile, for a whole warp or for one thread: the first is worked
    // out on the spot, the others come through the queue.
    auto take_tile = [&](int j) {
        if (j == 0) return find_tile(g, live, first);
        const int slot = (j - 1) % kQueue;
        Tile t;
        ok = tc::mbar_wait(queue_full + 8 * slot, ((j - 1) / kQueue) & 1);
        const int4 x = *reinterpret_cast<const int4*>(queue + slot);
        const int2 y = *reinterpret_cast<const int2*>(&queue[slot].kb);
        t.w = x.x, t.m = x.y, t.n = x.z, t.s = x.w, t.kb = y.x, t.ke = y.y;
        return t;
    };
    auto tile_taken = [&](int j) {  // one thread
        if (j > 0) tc::mbar_arrive_cluster(tc::map_to_rank(queue_empty + 8 * ((j - 1) % kQueue), 0));
    };

    if (warp == 0 && lane == 0) {
        int it = 0;
        for (int j = 0;; ++j) {
            const Tile t = take_tile(j);
            if (!ok || t.w < 0) break;
            tile_taken(j);
            const Work& x = g.work[t.w];
            const CUtensorMap *map_a = &maps.a[t.w], *map_b = &maps.b[t.w];
            const bool a_mn = x.product == kHead, b_mn = x.product >= kHead;
            const int am = t.m * kTile + (int)rank * kHalf;
            const int bn = t.n * kTile + (int)rank * kHalf + (b_mn ? 0 : x.v0);
            const int bk = x.product == kHidden ? x.v0 : 0;
            for (int k = t.kb; k < t.ke; ++k, ++it) {
                const int st = it % kStages;
                const uint32_t a = smem + st * kStageBytes, b = a + kHalf * kBlockK * 2;
                ok = tc::mbar_wait(empty + 8 * st, ((it / kStages) & 1) ^ 1);
                if (!ok) break;
                const uint32_t bar = tc::map_to_rank(full + 8 * st, 0);
                if (rank == 0) tc::mbar_expect_tx(full + 8 * st, 2 * kStageBytes);
                if (a_mn) {
                    tc::tma_load_2d(a, map_a, am, k * kBlockK, bar);
                    tc::tma_load_2d(a + 8192, map_a, am + 64, k * kBlockK, bar);
                } else {
                    tc::tma_load_2d(a, map_a, k * kBlockK, am, bar);
                }
                if (b_mn) {
                    tc::tma_load_2d(b, map_b, bn, bk + k * kBlockK, bar);
                    tc::tma_load_2d(b + 8192, map_b, bn + 64, bk + k * kBlockK, bar);
                } else {
                    tc::tma_load_2d(b, map_b, k * kBlockK, bn, bar);
                }
            }
            if (!ok) break;
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        int it = 0;
        for (int j = 0;; ++j) {
            const Tile t = take_tile(j);
            if (!ok || t.w < 0) break;
            tile_taken(j);
            const int product = g.work[t.w].product;
            const bool a_mn = product == kHead, b_mn = product >= kHead;
            const uint32_t idesc = tc::instr_desc(kTile, kTile, a_mn, b_mn);
            // K-major: 16 k are 32 bytes of every row; MN-major: two 8-column groups
            const uint32_t a_lbo = a_mn ? 8192 : 16, b_lbo = b_mn ? 8192 : 16;
            const uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
            const uint32_t d = tmem + (j & 1) * kTile;
            ok = tc::mbar_wait(acc_empty + 8 * (j & 1), ((j >> 1) & 1) ^ 1);
            if (!ok) break;
            tc::fence_after();
            for (int k = t.kb; k < t.ke; ++k, ++it) {
                const int st = it % kStages;
                ok = tc::mbar_wait(full + 8 * st, (it / kStages) & 1);
                if (!ok) break;
                tc::fence_after();
                const uint32_t a = smem + st * kStageBytes, b = a + kHalf * kBlockK * 2;
                const uint64_t da = tc::operand_desc(a, a_lbo, 1024), db = tc::operand_desc(b, b_lbo, 1024);
#pragma unroll
                for (int i = 0; i < kBlockK / 16; ++i)
                    tc::mma_pair(d, da + i * a_step, db + i * b_step, idesc, k > t.kb || i > 0);
                tc::commit_pair(empty + 8 * st);
            }
            if (!ok) break;
            tc::commit_pair(acc_full + 8 * (j & 1));
        }
    } else if (warp == 2 && lane == 0 && first == 0 && rank == 0 && g.expire) {
        ok = tc::mbar_wait(never, 0);
    } else if (warp == 3 && lane == 0 && rank == 0) {
        for (int j = 0; first < total_tiles(g, live); ++j) {
            const int slot = j % kQueue;
            ok = tc::mbar_wait<true>(queue_empty + 8 * slot, ((j / kQueue) & 1) ^ 1);
            if (!ok) break;
            const Tile t = find_tile(g, live, pairs + atomicAdd(g.next, 1));
            for (uint32_t r = 0; r < 2; ++r) {
                const uint32_t at = tc::map_to_rank(tc::smem_addr(queue + slot), r);
                const uint32_t bar = tc::map_to_rank(queue_full + 8 * slot, r);
                tc::mbar_expect_tx_cluster(bar, sizeof(Tile));
                tc::st_async(at, bar, t.w, t.m, t.n, t.s);
                tc::st_async(at + 16, bar, t.kb, t.ke, 0, 0);
            }
            if (t.w < 0) break;
        }
    } else if (warp == 3 && rank == 1 && first == 0 && g.partials) {
        sum_losses(g.partials, g.n_partials, live, g.mean, g.loss);
        __threadfence();
        if (lane == 0 && *static_cast<volatile int*>(&g.header->failed)) *static_cast<volatile float*>(g.loss) = NAN;
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t acc_empty0 = tc::map_to_rank(acc_empty, 0);
        const float scale = g.header->scale;
        for (int j = 0;; ++j) {
            const Tile t = take_tile(j);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok || t.w < 0) break;
            __syncwarp();  // every lane's read of the queue before the slot is given back
            if (lane == 0) tile_taken(j);
            const Work& x = g.work[t.w];
            const int row0 = t.m * kTile + (int)rank * kHalf + quad * 32, row = row0 + lane;
            const int col0 = t.n * kTile + half * kColumns;
            const uint32_t d = tmem + (j & 1) * kTile + half * kColumns + ((uint32_t)quad << 21);
            ok = tc::mbar_wait(acc_full + 8 * (j & 1), (j >> 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc::fence_after();
            // 32 columns at a time; but for the statistics, which are bound by their arithmetic and
            // gain nothing, the next ones are on their way while these are worked on (292 x 6382 x
            // 3584: 113.7 -> 103.8 us)
            uint32_t r[2][32];
            tc::tmem_ld32(d, r[0]);
            if (x.product <= kProbability) {
                const int y = row < live ? g.target[row] - (x.v0 + col0) : -1;  // column of the target
                const int left = g.vocab - (x.v0 + col0);                       // columns that exist
                if (x.product == kStatistics) {
                    // the target's own exponential is left out: it is added from a logit of its own
                    float top = -INFINITY, sum = 0.f;
#pragma unroll 1
                    for (int c = 0; c < kColumns && c < left; c += 32) {
                        __syncwarp();
                        if (c > 0) tc::tmem_ld32(d + c, r[0]);
                        tc::tmem_wait(r[0]);
                        if (c + 32 > left) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[0][i] = c + i < left ? r[0][i] : __float_as_uint(-INFINITY);
                        }
                        if (y >= c && y < c + 32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[0][i] = c + i == y ? __float_as_uint(-INFINITY) : r[0][i];
                        }
                        add_logits(r[0], g.log2e, top, sum);
                    }
                    if (row < live) g.stats[(int64_t)(2 * t.n + half) * g.rows + row] = make_float2(top, sum);
                } else {
                    const float2 rl = row < live ? g.row_loss[row] : make_float2(0.f, 0.f);
                    uint16_t* o = x.p + (int64_t)row * x.ldp + col0;
#pragma unroll 1
                    for (int c = 0; c < kColumns; c += 64) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = c + 32 * h;
                            __syncwarp();
                            tc::tmem_wait(r[h]);
                            if (at + 32 < kColumns) tc::tmem_ld32(d + at + 32, r[h ^ 1]);
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = ss::pack_bf16x2(ex2(fmaf(__uint_as_float(r[h][2 * i]), g.log2e, -rl.x)),
                                                       ex2(fmaf(__uint_as_float(r[h][2 * i + 1]), g.log2e, -rl.x)));
                            if (row >= live || at + 32 > left) {  // zeros where there is no token or no class
                                const int have = row < live ? left - at : 0;
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    w[i] = 2 * i + 1 < have ? w[i] : 2 * i < have ? w[i] & 0xFFFFu : 0u;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<uint4*>(o + at + 8 * i) =
                                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                        }
                    }
                    if (y >= 0 && y < kColumns && y < left) o[y] = ss::f32_to_bf16(rl.y);  // over its exponential
                }
            } else {
                // through shared memory (16-byte groups of row i at group ^ (i & 7), free of bank
                // conflicts both ways), so that a row's values go out together
                const int limit = x.product == kHidden ? live : x.m_rows;
                const int* token = x.product == kHidden ? g.token : nullptr;
                const bool none = t.kb == t.ke;  // no k: the accumulator holds something else
                float* mine = turn[warp - 4];
                uint32_t* words = reinterpret_cast<uint32_t*>(mine);
                const int k = lane & 7;
                if (x.part) {  // fp32, 32 columns at a time: 8 lanes a row, 4 columns a lane
                    float* part = x.part + t.s * x.part_split + (int64_t)(row0 + (lane >> 3)) * x.part_ld + col0 + 4 * k;
#pragma unroll 1
                    for (int c = 0; c < kColumns && col0 + c < x.cols; c += 64) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = c + 32 * h;
                            __syncwarp();
                            tc::tmem_wait(r[h]);
                            if (at + 32 < kColumns) tc::tmem_ld32(d + at + 32, r[h ^ 1]);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4*>(words + lane * 32 + 4 * (i ^ (lane & 7))) =
                                    none ? make_uint4(0, 0, 0, 0)
                                         : make_uint4(r[h][4 * i], r[h][4 * i + 1], r[h][4 * i + 2], r[h][4 * i + 3]);
                            __syncwarp();
                            if (col0 + at + 4 * k >= x.cols) continue;  // part_ld is a multiple of 4
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int q = 4 * i + (lane >> 3);
                                if (row0 + q >= limit) continue;
                                float4 v = *reinterpret_cast<const float4*>(mine + q * 32 + 4 * (k ^ (q & 7)));
                                float4* o = reinterpret_cast<float4*>(part + (int64_t)(4 * i) * x.part_ld + at);
                                if (x.add) {
                                    const float4 w = *o;
                                    v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                                }
                                *o = v;
                            }
                        }
                    }
                } else if ((reinterpret_cast<uintptr_t>(x.out) & 15u) == 0 && (x.out_ld & 7) == 0) {
                    // bf16 rows on 16-byte boundaries, 64 columns at a time: 8 lanes a row, 16 bytes a lane
#pragma unroll 1
                    for (int c = 0; c < kColumns && col0 + c < x.cols; c += 64) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = c + 32 * h;
                            __syncwarp();
                            tc::tmem_wait(r[h]);
                            if (at + 32 < kColumns) tc::tmem_ld32(d + at + 32, r[h ^ 1]);
                            turn_words(words, lane, h, r[h], scale, none);
                        }
                        __syncwarp();
                        const int col = col0 + c + 8 * k, left = x.cols - col;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int q = 4 * i + (lane >> 3);
                            if (row0 + q >= limit || left <= 0) continue;
                            const int64_t orow = token ? token[row0 + q] : (int64_t)x.v0 + row0 + q;
                            uint16_t* o = x.out + orow * x.out_ld + col;
                            const uint4 v = *reinterpret_cast<const uint4*>(words + q * 32 + 4 * (k ^ (q & 7)));
                            if (left >= 8)
                                *reinterpret_cast<uint4*>(o) = v;
                            else
                                ss::st_bytes(reinterpret_cast<unsigned char*>(o), v, 0, 2 * left);
                        }
                    }
                } else {
                    // bf16 rows at any element offset, 64 columns at a time.  Of a row's 128 bytes the 7
                    // aligned blocks inside go out as such, put together from two groups, and the 8
                    // elements before and after them one a lane; a row's last columns word by word.
                    // (All of them word by word: 230 us where this takes 205, 604 of 1021 tokens, 32003 x 1001.)
#pragma unroll 1
                    for (int c = 0; c < kColumns && col0 + c < x.cols; c += 64) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            __syncwarp();
                            if (c + h > 0) tc::tmem_ld32(d + c + 32 * h, r[0]);
                            tc::tmem_wait(r[0]);
                            turn_words(words, lane, h, r[0], scale, none);
                        }
                        __syncwarp();
                        const int col = col0 + c, left = x.cols - col;
                        const int here = min(limit - row0, 32);
                        if (left >= 64) {
#pragma unroll 4
                            for (int i = 0; i < 8; ++i) {
                                const int q = 4 * i + (lane >> 3);
                                if (q >= here) continue;
                                const int64_t orow = token ? token[row0 + q] : (int64_t)x.v0 + row0 + q;
                                uint16_t* o = x.out + orow * x.out_ld + col;
                                const int sh = (int)(reinterpret_cast<uintptr_t>(o) & 15u);
                                const uint32_t* row_q = words + q * 32;
                                const uint4 mine4 = *reinterpret_cast<const uint4*>(row_q + 4 * (k ^ (q & 7)));
                                const uint4 next4 = *reinterpret_cast<const uint4*>(row_q + 4 * (min(k + 1, 7) ^ (q & 7)));
                                if (sh == 0) {
                                    *reinterpret_cast<uint4*>(o + 8 * k) = mine4;
                                    continue;
                                }
                                if (k < 7)
                                    *reinterpret_cast<uint4*>(o + 8 * k + 8 - sh / 2) = ss::realign16(mine4, next4, 16 - sh);
                                const int e = 2 * k < 16 - sh ? k : 56 + k;  // before the blocks, or after
                                const uint32_t w = row_q[4 * ((e >> 3) ^ (q & 7)) + ((e & 7) >> 1)];
                                o[e] = (uint16_t)(e & 1 ? w >> 16 : w);
                            }
                        } else {
                            for (int q = 0; q < here; ++q) {
                                const int64_t orow = token ? token[row0 + q] : (int64_t)x.v0 + row0 + q;
                                uint16_t* o = x.out + orow * x.out_ld + col;
                                const uint32_t w = words[q * 32 + 4 * ((lane >> 2) ^ (q & 7)) + (lane & 3)];
                                if (2 * lane < left) o[2 * lane] = (uint16_t)w;
                                if (2 * lane + 1 < left) o[2 * lane + 1] = (uint16_t)(w >> 16);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            tc::tmem_wait(r[0]);  // a load asked for and not used
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_cluster(acc_empty0 + 8 * (j & 1));
        }
    }
    if (!ok) {
        give_up(g.header, g.loss);
        // copies in flight land before the CTA goes: those that its other roles have asked for since (this
        // one's own are two seconds old)
        const uint64_t t0 = tc::global_ns();
        while (tc::global_ns() - t0 < 1000000ull) __nanosleep(20000);
    }
    __syncwarp();
    tc::fence_before();
    tc::cluster_sync();
    tc::fence_after();
    if (warp == 2) tc::tmem_free(tmem, 512);
}

// ---------------------------------------------------------------------------
// around the products
// ---------------------------------------------------------------------------

constexpr int kThreads = 256;
constexpr int kGatherRows = 8;  // tokens per CTA, one per warp
constexpr int kGatherThreads = 32 * kGatherRows;

// 8 elements from element 8j of a row of D bf16 at any element alignment,
// zeros past its end.
__device__ __forceinline__ uint4 row_vec(const uint16_t* row, int j, int D) {
    if (8 * j + 8 <= D) return ss::ld_any16(row + 8 * j);
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 8 * j; i < D; ++i) w[(i & 7) >> 1] |= (uint32_t)row[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float dot_bf16(uint4 a, uint4 b, float s) {
    s = fmaf(ss::bf16_lo(a.x), ss::bf16_lo(b.x), s);
    s = fmaf(ss::bf16_hi(a.x), ss::bf16_hi(b.x), s);
    s = fmaf(ss::bf16_lo(a.y), ss::bf16_lo(b.y), s);
    s = fmaf(ss::bf16_hi(a.y), ss::bf16_hi(b.y), s);
    s = fmaf(ss::bf16_lo(a.z), ss::bf16_lo(b.z), s);
    s = fmaf(ss::bf16_hi(a.z), ss::bf16_hi(b.z), s);
    s = fmaf(ss::bf16_lo(a.w), ss::bf16_lo(b.w), s);
    return fmaf(ss::bf16_hi(a.w), ss::bf16_hi(b.w), s);
}

struct GatherArgs {
    Header* header;
    const int64_t* targets;
    int64_t ignore;
    int T, D, Dp, vocab;
    const uint16_t* hidden;
    int64_t ld;
    const uint16_t* weight;
    int64_t ldw;
    uint16_t* h;          // [rows][Dp]
    int* row;             // [rows]: token of each gathered row
    int* target;          // [rows]
    float* target_logit;  // [rows]
    float* token_loss;    // nullable
    uint16_t* d_hidden;   // nullable
    int64_t d_ld;
    float grad_scale;
    int mean;
    int* counters;  // of the launches' tiles
    int n_counters;
    const int* chunk;  // tokens that count in each kChunk of them (NULL: count one by one)
};

// From so many tokens on, ce_count_kernel counts them by chunks first.  Counting one
// by one reads T * T / 2 bytes from L2 in all: 130 MB for 16384 tokens, a few us, but
// 0.5 TB for a million.
constexpr int kChunk = 2048;
constexpr int64_t kChunksFrom = 16384;

__global__ void __launch_bounds__(kGatherThreads) ce_count_kernel(const int64_t* targets, int64_t ignore, int T, int* chunk) {
    __shared__ int part[kGatherThreads / 32];
    wait_before();
    launch_after();
    const int t0 = blockIdx.x * kChunk;
    int n = 0;
#pragma unroll
    for (int i = threadIdx.x; i < kChunk; i += kGatherThreads) n += t0 + i < T && targets[t0 + i] != ignore;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        n = 0;
        for (int i = 0; i < kGatherThreads / 32; ++i) n += part[i];
        chunk[blockIdx.x] = n;
    }
}

// Block b places tokens [8 b, 8 b + 8): how many of the tokens before count
// (by chunks where they have been counted; read again by every block), then its own
// rows, one per warp: gathered together with the logit of their target, or,
// where ignored, zeroed in the outputs.  The target's logit is the one that grows
// large, and the tensor cores' sums drop bits in one direction (kDropped), so it
// gets a sum of its own, in fp32 by 256 partial sums.  The last block knows the total.
__device__ __forceinline__ void gather_block(const GatherArgs& a, int block, bool last) {
    __shared__ int part[kGatherRows];
    __shared__ int flag[kGatherRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = block * kGatherRows;
    const int t = t0 + warp;
    const int64_t y = t < a.T ? a.targets[t] : a.ignore;
    const bool counts = y != a.ignore, known = y >= 0 && y < a.vocab;
    const uint16_t* src = a.hidden + (int64_t)t * a.ld;
    const uint16_t* w = a.weight + (known ? y : 0) * a.ldw;
    if (counts) {  // both rows on their way to L2 while the tokens before are counted
        for (int j = 64 * lane; j < a.D; j += 64 * 32) {
            ss::prefetch_l2(src + j);
            ss::prefetch_l2(w + j);
        }
    }
    int before = 0;
    const int chunks = a.chunk ? t0 / kChunk : 0;
    for (int i = threadIdx.x; i < chunks; i += kGatherThreads) before += a.chunk[i];
#pragma unroll 8
    for (int i = chunks * kChunk + threadIdx.x; i < t0; i += kGatherThreads) before += a.targets[i] != a.ignore;
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (lane == 0) part[warp] = before, flag[warp] = counts;
    __syncthreads();
    const int sum = __reduce_add_sync(0xFFFFFFFFu, lane < kGatherRows ? part[lane] : 0);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, lane < kGatherRows && flag[lane]);
    const int vecs = a.Dp / 8;
    if (counts) {
        const int at = sum + __popc(mask & ((1u << warp) - 1));
        uint4* dst = reinterpret_cast<uint4*>(a.h + (int64_t)at * a.Dp);
        float s = 0.f;
#pragma unroll 4
        for (int j = lane; j < vecs; j += 32) {
            const uint4 x = row_vec(src, j, a.D);
            dst[j] = x;
            s += dot_bf16(x, row_vec(w, j, a.D), 0.f);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        if (lane == 0) {
            a.row[at] = t;
            a.target[at] = known ? (int)y : -1;
            a.target_logit[at] = known ? s : NAN;
        }
    } else if (t < a.T) {
        if (lane == 0 && a.token_loss) a.token_loss[t] = 0.f;
        if (a.d_hidden) {
            uint16_t* dst = a.d_hidden + (int64_t)t * a.d_ld;
            for (int j = lane; j < a.D; j += 32) dst[j] = 0;
        }
    }
    if (last) {
        for (int i = threadIdx.x; i < a.n_counters; i += kGatherThreads) a.counters[i] = 0;
        if (threadIdx.x == 0) {
            const int live = sum + __popc(mask);
            a.header->live = live;
            a.header->finished = 0;
            a.header->failed = 0;
            a.header->scale = a.mean ? (live > 0 ? a.grad_scale / (float)live : 0.f) : a.grad_scale;
        }
    }
}

__global__ void __launch_bounds__(kGatherThreads) ce_gather_kernel(const GatherArgs a) {
    wait_before();
    launch_after();  // only now: ce_stage_kernel reads and writes before its own wait
    gather_block(a, blockIdx.x, blockIdx.x == gridDim.x - 1);
}

// Rows of a weight whose rows do not start on 16-byte boundaries, copied to
// rows that do: one warp per row.  It needs nothing of the gather, and only ends
// after it, for the kernels behind both; as the first kernel of a call it waits at once.
__global__ void __launch_bounds__(kThreads)
ce_stage_kernel(const uint16_t* __restrict__ w, int64_t ld, int V, int D, int Dp, int first,
                uint16_t* __restrict__ out) {
    if (first) wait_before();
    launch_after();
    const int lane = threadIdx.x & 31;
    const int64_t v = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (v < V) {  // a lane's aligned 16 bytes and its neighbour's make its vector
        const uint16_t* src = w + v * ld;
        const int sh = (int)(reinterpret_cast<uintptr_t>(src) & 15u);
        const unsigned char* base = reinterpret_cast<const unsigned char*>(src) - sh;
        const int blocks = (sh + 2 * D + 15) / 16, vecs = Dp / 8;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        uint4* dst = reinterpret_cast<uint4*>(out + v * Dp);
        for (int j0 = lane; j0 < vecs + lane; j0 += 128) {  // four loads of a lane before the first is used
            uint4 x[4], e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = j0 + 32 * i;
                x[i] = j < blocks ? ss::ld_stream_u4(base + 16 * j) : zero;
                e[i] = lane == 31 && j + 1 < blocks ? ss::ld_stream_u4(base + 16 * (j + 1)) : zero;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = j0 + 32 * i;
                uint4 y;
                y.x = __shfl_down_sync(0xFFFFFFFFu, x[i].x, 1), y.y = __shfl_down_sync(0xFFFFFFFFu, x[i].y, 1);
                y.z = __shfl_down_sync(0xFFFFFFFFu, x[i].z, 1), y.w = __shfl_down_sync(0xFFFFFFFFu, x[i].w, 1);
                if (lane == 31) y = e[i];
                uint4 r = sh ? ss::realign16(x[i], y, sh) : x[i];
                if (8 * j + 8 > D) {  // zeros past the row's end
                    uint32_t q[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (8 * j + k >= D) q[k >> 1] &= (k & 1) ? 0x0000FFFFu : 0xFFFF0000u;
                    r = make_uint4(q[0], q[1], q[2], q[3]);
                }
                if (j < vecs) dst[j] = r;
            }
        }
    }
    wait_before();
}

// ---------------------------------------------------------------------------
// statistics of a few tokens
// ---------------------------------------------------------------------------

// With a handful of tokens the weight's one read is all the time there is: dot
// products on the CUDA cores against the tokens in shared memory, 8 loads in flight a
// lane: of 2 weight rows, and from 3 tokens on, where shared memory is what is read
// most (a token's vector once for all rows), of 4.
// Against the tile kernel, with vocabulary and hidden size 32000 x 2048, 32000 x 4096
// and 5000 x 512: 1 or 2 tokens 28-30, 49-52 and 11 us (42, 68, 14), 3 or 4 tokens 35,
// 54 and 11; from 5 on the tiles win (42 against 42, 68 against 71 with dot products).
constexpr int kFewTokens = 4;
constexpr int kFewLoads = 8;
constexpr int kFewSmem = 64 * 1024;  // of hidden states
constexpr int few_rows(int64_t tokens) { return tokens <= 2 ? 2 : 4; }
// CTAs per SM at most, each a slice of statistics; their registers allow no more
constexpr int few_ctas_per_sm(int64_t tokens) { return tokens <= 2 ? 4 : 2; }

// Bound by the weight's read: 131 MB in 26 us at 32000 x 2048, 65 % of the DRAM's
// rate; the launch's start and its last round are the rest.  One token: 4 CTAs of 8
// warps an SM measured 28.2 us a call, 3 and 5 of them 29.5; one row a warp 29.2, 4 rows
// 28.2 (20.5 for 19.7 at 50000 x 768), 16 loads in flight 28.7 to 35, loads through a
// ring in shared memory, always 12 in flight, 31 to 35.  4 tokens: 2 rows a warp 41.1, 4
// rows 35.1, 8 rows 55; as many CTAs as with one token 36.8.
//
// Statistics as the tile kernel leaves them, one slice per CTA: CTA b's warps
// take groups of ROWS rows, b's after those of the CTA before.  The CTAs pick
// the tokens that count out themselves; one more CTA does the gather's work for
// the kernels behind.
template <int TOKENS, int ROWS>
__global__ void __launch_bounds__(kThreads)
ce_few_kernel(const GatherArgs a, const uint16_t* __restrict__ w, int64_t ldw, int rows, float2* stats) {
    launch_after();
    wait_before();
    if (blockIdx.x == gridDim.x - 1) {
        gather_block(a, 0, true);
        return;
    }
    extern __shared__ __align__(16) unsigned char raw[];
    uint4* hs = reinterpret_cast<uint4*>(raw);
    __shared__ float top_s[kThreads / 32][kFewTokens];
    __shared__ float sum_s[kThreads / 32][kFewTokens];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // whole vectors of a row and the elements behind them, which go by themselves: what lies
    // between a row's end and the next one's start, or behind the last row, may be a NaN
    const int vecs = a.D / 8, rest = a.D % 8, ld_hs = (a.D + 7) / 8;
    const int V = a.vocab, slices = gridDim.x - 1;
    const int groups = (V + ROWS - 1) / ROWS;
    int g = blockIdx.x * (kThreads / 32) + warp;
    constexpr int U = kFewLoads / ROWS;  // of each row
    uint4 x[U][ROWS];
    auto load = [&](int g, int j) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {  // past the end: the last row again, left out below
            const int v = g * ROWS + r < V ? g * ROWS + r : V - 1;
            const uint4* p = reinterpret_cast<const uint4*>(w + (int64_t)v * ldw);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (j + 32 * i < vecs) x[i][r] = ss::ld_stream_u4(p + j + 32 * i);
        }
    };
    bool loaded = g < groups && lane < vecs;  // the first loads go out before the tokens are known
    if (loaded) load(g, lane);
    int y[TOKENS], from[TOKENS], live = 0;  // target and token of each row
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) y[t] = -1, from[t] = -1;
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
        const int64_t target = t < a.T ? a.targets[t] : a.ignore;
        if (target == a.ignore) continue;
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) {
            if (i != live) continue;
            y[i] = target >= 0 && target < V ? (int)target : -1;
            from[i] = t;
        }
        ++live;
    }
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
        for (int j = threadIdx.x; j < ld_hs; j += kThreads)
            hs[t * ld_hs + j] = from[t] >= 0 ? row_vec(a.hidden + from[t] * a.ld, j, a.D) : make_uint4(0, 0, 0, 0);
    __syncthreads();
    float top[TOKENS], sum[TOKENS];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) top[t] = -INFINITY, sum[t] = 0.f;
    for (; g < groups; g += slices * (kThreads / 32)) {
        const int v0 = g * ROWS;
        float acc[ROWS][TOKENS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) acc[r][t] = 0.f;
        for (int j = lane; j < vecs; j += 32 * U) {
            if (j != lane || !loaded) load(g, j);
            loaded = false;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (j + 32 * i >= vecs) continue;
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    const uint4 hv = hs[t * ld_hs + j + 32 * i];
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) acc[r][t] = dot_bf16(x[i][r], hv, acc[r][t]);
                }
            }
        }
        __syncwarp();
        if (lane < rest) {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(hs) + 8 * vecs + lane;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float wv = ss::bf16_to_f32(w[(int64_t)min(v0 + r, V - 1) * ldw + 8 * vecs + lane]);
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) acc[r][t] = fmaf(wv, ss::bf16_to_f32(h[8 * t * ld_hs]), acc[r][t]);
            }
        }
        const int next = g + slices * (kThreads / 32);  // its loads go out before this group's sums
        loaded = next < groups && lane < vecs;
        if (loaded) load(next, lane);
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            float l[ROWS], m = -INFINITY;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                l[r] = acc[r][t];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], d);
                if (v0 + r >= V || v0 + r == y[t]) l[r] = -INFINITY;
                m = fmaxf(m, l[r]);
            }
            const float up = fmaxf(top[t], ceilf(m * kLog2e));
            const float at = up == -INFINITY ? 0.f : up;
            float a = 0.f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) a += ex2(fmaf(l[r], kLog2e, -at));
            sum[t] = (top[t] == -INFINITY ? sum[t] : sum[t] * ex2(top[t] - at)) + a;  // as in add_logits
            top[t] = up;
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) top_s[warp][t] = top[t], sum_s[warp][t] = sum[t];
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < TOKENS && t < live) {
        float m = -INFINITY, s = 0.f;
        for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, top_s[i][t]);
        const float at = m == -INFINITY ? 0.f : m;
        for (int i = 0; i < kThreads / 32; ++i)
            s += top_s[i][t] == -INFINITY ? sum_s[i][t] : sum_s[i][t] * ex2(top_s[i][t] - at);
        stats[(int64_t)blockIdx.x * rows + t] = make_float2(m, s);
    }
}

constexpr int kLossThreads = 256;
constexpr int kLossRows = kLossThreads / 32;  // rows per CTA, 32 threads each
constexpr int kLossSlices = 32;

// The tiles' statistics of a row to its loss.  With r = sum over every other
// class of exp(l - l_target): loss = log(1 + r), log-sum-exp = l_target + loss and
// the target's p - 1 = -r / (1 + r), none of which cancels where the target holds
// almost all of the mass.  The CTA's losses go to one fp64 partial.  With no
// gradient to follow, the last CTA to finish sums the partials (sum_losses); else
// the next launch does, off the gradients' path, and h is given: the gathered hidden
// states are zeroed from the last row to the next whole k block.  Where the statistics
// gave up, every token's loss is NaN, and so are the loss and the gradients made of it.
__global__ void __launch_bounds__(kLossThreads)
ce_loss_kernel(Header* header, const float2* __restrict__ stats, int n_tiles, int rows,
               const float* __restrict__ target_logit, const int* __restrict__ row_map,
               float2* __restrict__ row_loss, float* __restrict__ token_loss, double* __restrict__ partials,
               int mean, float* __restrict__ loss_out, uint16_t* h, int Dp) {
    launch_after();
    __shared__ float top_s[kLossSlices][kLossRows + 1];
    __shared__ float sum_s[kLossSlices][kLossRows + 1];
    __shared__ double loss_s[kLossRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_before();
    const int live = header->live;
    auto add = [](float& m, float& s, float m2, float s2) {  // exponents are whole numbers: exact
        const float up = fmaxf(m, m2);
        s = (m == up ? s : s * ex2(m - up)) + (m2 == up ? s2 : s2 * ex2(m2 - up));
        m = up;
    };
    {  // rows side by side, a thread's slice of the tiles
        const int r = threadIdx.x % kLossRows, slice = threadIdx.x / kLossRows;
        const int row = blockIdx.x * kLossRows + r;
        float top = -INFINITY, sum = 0.f;
        if (row < live) {
            int n = slice;
            for (; n < n_tiles; n += 8 * kLossSlices) {
                float2 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = n + i * kLossSlices < n_tiles ? stats[(int64_t)(n + i * kLossSlices) * rows + row]
                                                         : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) add(top, sum, v[i].x, v[i].y);
            }
        }
        top_s[slice][r] = top;
        sum_s[slice][r] = sum;
    }
    const int row = blockIdx.x * kLossRows + warp;  // from here on a warp's row, a lane's slice
    if (h && row >= live && row < (live + kBlockK - 1) / kBlockK * kBlockK)
        for (int j = lane; j < Dp / 8; j += 32) reinterpret_cast<uint4*>(h + (int64_t)row * Dp)[j] = make_uint4(0, 0, 0, 0);
    const float hit = row >= live ? 0.f : header->failed ? NAN : target_logit[row];
    const int token = row < live ? row_map[row] : 0;
    __syncthreads();
    float top = top_s[lane][warp], sum = sum_s[lane][warp];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
        add(top, sum, __shfl_xor_sync(0xFFFFFFFFu, top, k), __shfl_xor_sync(0xFFFFFFFFu, sum, k));
    if (lane == 0) {
        float l = 0.f;
        if (row < live) {
            // log of r, the whole exponent's ln 2 in two parts (the first exact); a lone class has r = 0
            const float low = fmaf(top, kLn2Low, logf(sum));
            float d = top == -INFINITY ? (sum == 0.f ? top : sum) : fmaf(top, kLn2High, -hit) + low;
            // no loss without a target's logit, with one of +inf (inf - inf), or with nothing but -inf
            if (!(hit < INFINITY) || (hit == -INFINITY && d == -INFINITY)) d = NAN;
            const float rest = expf(-fabsf(d));
            l = (d > 0.f ? d : 0.f) + log1pf(rest);
            // of a target at -inf the loss is infinite, and log-sum-exp what the other classes have
            const float lse = hit == -INFINITY ? fmaf(top, kLn2High, low) : hit + l;
            row_loss[row] = make_float2(lse * kLog2e, -(d > 0.f ? 1.f : rest) / (1.f + rest));
            if (token_loss) token_loss[token] = l;
        }
        loss_s[warp] = (double)l;
    }
    __syncthreads();
    if (warp == 0) {
        double loss = lane < kLossRows ? loss_s[lane] : 0.0;
#pragma unroll
        for (int k = kLossRows / 2; k > 0; k >>= 1) loss += __shfl_down_sync(0xFFFFFFFFu, loss, k);
        if (lane == 0) partials[blockIdx.x] = loss;
        if (h) return;
        int last = 1;
        if (gridDim.x > 1) {
            if (lane == 0) {
                __threadfence();
                last = atomicAdd(&header->finished, 1) == (int)gridDim.x - 1;
                __threadfence();
            }
            last = __shfl_sync(0xFFFFFFFFu, last, 0);
        }
        __syncwarp();
        if (last) sum_losses(partials, gridDim.x, live, mean, loss_out);
    }
}

// out = bf16(scale * sum of the splits' partials), rows through row_map.
__global__ void __launch_bounds__(kThreads)
ce_join_kernel(const Header* __restrict__ header, const float* part, int splits, int64_t part_split,
               int part_ld, int rows, int cols, uint16_t* __restrict__ out, int64_t out_ld,
               const int* __restrict__ row_map) {
    launch_after();
    wait_before();
    const int limit = row_map ? header->live : rows;
    const int vecs = part_ld / 4;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t row = i / vecs;
    const int col = (int)(i % vecs) * 4;
    if (row >= limit) return;
    const float* p = part + row * part_ld + col;
    float4 s = *reinterpret_cast<const float4*>(p);
#pragma unroll 8
    for (int k = 1; k < splits; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(p + k * part_split);
        s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
    }
    const float c = header->scale;
    uint16_t* o = out + (row_map ? (int64_t)row_map[row] : row) * out_ld + col;
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < cols) o[e] = ss::f32_to_bf16(c * v[e]);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Splits of k that keep the pairs busy, by the clocks of each choice: a k block
// of a 256 x 256 tile takes a pair 512, and a tile's fp32 partial, written and
// read once, 512 KB at about 3500 bytes a clock.
int choose_splits(int64_t tiles, int64_t kblocks, int pairs) {
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 32 && (s == 1 || s * 4 <= kblocks); ++s) {
        const double rounds = (double)((tiles * s + pairs - 1) / pairs);
        const double cost = rounds * (double)((kblocks + s - 1) / s) * 512 + (s > 1 ? tiles * s * 150.0 : 0.0);
        if (cost < least) least = cost, best = s;
    }
    return best;
}

// Where everything lies in the workspace.
struct Layout {
    int64_t T, D, V, Dp, rows, n_tiles, slices, piece, pieces;
    bool few;  // tokens: the dot-product kernel
    int hidden_splits, head_splits;
    bool grad, stage;
    int64_t counters, n_counters, chunk;
    int64_t row, target, target_logit, row_loss, partials, stats, h, w, p[2], hidden_part, head_part, bytes;
};

constexpr int64_t kPieceBytes = 256ll << 20;  // of P, one buffer of two

Layout plan_layout(int64_t T, int64_t D, int64_t V, bool grad, bool stage, int pairs) {
    Layout l = {};
    l.T = T, l.D = D, l.V = V, l.grad = grad, l.stage = stage;
    l.Dp = up(D, 16);  // rows on 32-byte sectors
    l.rows = up(T, kTile);
    l.n_tiles = up(V, kTile) / kTile;
    l.few = T > 0 && T <= kFewTokens && kFewTokens * l.Dp * 2 <= kFewSmem;
    const int64_t per_cta = few_rows(T) * (kThreads / 32), few_ctas = (V + per_cta - 1) / per_cta;
    const int64_t few_most = 2 * pairs * few_ctas_per_sm(T);
    l.slices = !l.few ? 2 * l.n_tiles : few_ctas < few_most ? few_ctas : few_most;
    int64_t at = 256;  // the header
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    l.row = take(l.rows * 4);
    l.target = take(l.rows * 4);
    l.target_logit = take(l.rows * 4);
    l.row_loss = take(l.rows * 8);
    l.partials = take(l.rows / kLossRows * 8);
    if (grad) {
        const int64_t fit = kPieceBytes / (l.rows > 0 ? l.rows * 2 : 2) / kTile * kTile;
        l.piece = fit < kTile ? kTile : fit;
        l.pieces = (l.n_tiles * kTile + l.piece - 1) / l.piece;
        l.piece = (l.n_tiles + l.pieces - 1) / l.pieces * kTile;  // even pieces
    }
    l.n_counters = 2 + l.pieces;
    l.counters = take(l.n_counters * 4);
    l.chunk = T >= kChunksFrom ? take(up(T, kChunk) / kChunk * 4) : 0;
    l.stats = take(l.slices * l.rows * 8);
    l.h = take(l.rows * l.Dp * 2);
    if (stage) l.w = take(V * l.Dp * 2);
    if (grad) {
        l.p[0] = take(l.rows * l.piece * 2);
        l.p[1] = l.pieces > 1 ? take(l.rows * l.piece * 2) : l.p[0];
        const int64_t d_tiles = up(D, kTile) / kTile;
        l.hidden_splits = choose_splits(l.rows / kTile * d_tiles, l.piece / kBlockK, pairs);
        l.head_splits = choose_splits(l.piece / kTile * d_tiles, l.rows / kBlockK, pairs);
        const int64_t ld = up(D, 4);
        if (l.hidden_splits > 1 || l.pieces > 1) l.hidden_part = take(l.hidden_splits * l.rows * ld * 4);
        if (l.head_splits > 1) l.head_part = take(l.head_splits * l.piece * ld * 4);
    }
    l.bytes = at;
    return l;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A [rows][cols] bf16 matrix of row stride ld, in boxes of 64 columns and
// box_rows rows, out-of-range elements read as zero.
int make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const EncodeTiled fn = encoder();
    if (!fn) return ss::cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SS_OK : ss::cuda_fail(cudaErrorInvalidValue);
}

// Launch chained to the kernel before it (see launch_after).
template <class K, class... A>
int launch(K kernel, int64_t grid, int threads, int smem, cudaStream_t st, A&&... args) {
    return ss::launch(kernel, grid, threads, smem, 0, true, st, args...);
}

// Raises a kernel's limit of dynamic shared memory, once for each device.
int allow_smem(std::atomic<uint64_t>& ready, const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return ss::cuda_fail(e);
    const uint64_t bit = 1ull << (dev & 63);
    if (ready.load(std::memory_order_acquire) & bit) return SS_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return ss::cuda_fail(e);
    if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
    return SS_OK;
}

template <int TOKENS>
int launch_few(const GatherArgs& a, const uint16_t* w, int64_t ldw, int64_t slices, int64_t rows,
               float2* stats, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    const auto kernel = ce_few_kernel<TOKENS, few_rows(TOKENS)>;
    if (int rc = allow_smem(ready, reinterpret_cast<const void*>(kernel), kFewSmem)) return rc;
    return launch(kernel, slices + 1, kThreads, TOKENS * a.Dp * 2, st, a, w, ldw, (int)rows, stats);
}

int launch_gemm(const Maps& maps, GemmArgs& g, int64_t tiles, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    if (int rc = allow_smem(ready, reinterpret_cast<const void*>(ce_gemm_kernel), kSmemBytes)) return rc;
    const int64_t pairs = ss::num_sms() / 2;
    const int rc = launch(ce_gemm_kernel, 2 * (tiles < pairs ? tiles : pairs), kGemmThreads, kSmemBytes, st, maps, g);
    ++g.next;
    return rc;
}

// The matrix launch of the next call that gets a wait which nothing ends (-1: none).
std::atomic<int> g_expire{-1};

constexpr int64_t kMaxSize = 1 << 28;  // tokens, hidden, vocabulary: 32-bit tile coordinates

bool valid_sizes(int64_t T, int64_t D, int64_t V) { return T >= 0 && D >= 1 && V >= 1; }

bool rows_aligned(const void* p, int64_t ld) { return ss::aligned(p, 16) && ld % 8 == 0; }

}  // namespace

extern "C" {

int ss_linear_ce_expire_wait(int launch) {
    if (launch < -1) return SS_EINVAL;
    g_expire.store(launch, std::memory_order_relaxed);
    return SS_OK;
}

int ss_linear_ce_workspace(int64_t num_tokens, int64_t hidden_size, int64_t vocab_size, unsigned flags,
                           size_t* bytes_out) {
    if (!bytes_out || !valid_sizes(num_tokens, hidden_size, vocab_size)) return SS_EINVAL;
    if (flags & ~(SS_CE_GRADIENT | SS_CE_STAGE_WEIGHT)) return SS_EINVAL;
    if (num_tokens > kMaxSize || hidden_size > kMaxSize || vocab_size > kMaxSize) return SS_EOVERFLOW;
    const bool stage = (flags & SS_CE_STAGE_WEIGHT) || hidden_size % 8 != 0;
    *bytes_out = (size_t)plan_layout(num_tokens, hidden_size, vocab_size, flags & SS_CE_GRADIENT, stage,
                                     ss::num_sms() / 2)
                     .bytes;
    return SS_OK;
}

int ss_linear_cross_entropy(const ss_linear_ce* a, ss_stream_t stream) {
    if (!a || !valid_sizes(a->num_tokens, a->hidden_size, a->vocab_size)) return SS_EINVAL;
    const int64_t T = a->num_tokens, D = a->hidden_size, V = a->vocab_size;
    if (T > kMaxSize || D > kMaxSize || V > kMaxSize) return SS_EOVERFLOW;
    if ((T > 0 && (!a->hidden || !a->targets)) || !a->weight || !a->loss_out || !a->workspace) return SS_EINVAL;
    if (a->reduction != SS_LOSS_MEAN && a->reduction != SS_LOSS_SUM) return SS_EINVAL;
    if (!std::isfinite((float)a->grad_scale)) return SS_EINVAL;  // it is used in fp32
    const bool grad = a->d_hidden || a->d_weight;
    if (a->hidden_stride < D || a->weight_stride < D || (a->d_hidden && a->d_hidden_stride < D) ||
        (a->d_weight && a->d_weight_stride < D))
        return SS_EINVAL;
    const int64_t most = INT64_MAX / 8;
    if (a->weight_stride > most / V || (T > 0 && a->hidden_stride > most / T) ||
        (a->d_weight && a->d_weight_stride > most / V) || (a->d_hidden && T > 0 && a->d_hidden_stride > most / T))
        return SS_EOVERFLOW;
    if (!ss::aligned(a->hidden, 2) || !ss::aligned(a->weight, 2) || !ss::aligned(a->d_hidden, 2) ||
        !ss::aligned(a->d_weight, 2) || !ss::aligned(a->targets, 8) || !ss::aligned(a->loss_out, 4) ||
        !ss::aligned(a->token_loss_out, 4) || !ss::aligned(a->workspace, 256))
        return SS_EALIGN;
    const bool stage = !rows_aligned(a->weight, a->weight_stride);
    const int pairs = ss::num_sms() / 2;
    const Layout l = plan_layout(T, D, V, grad, stage || D % 8 != 0, pairs);
    if (a->workspace_bytes < (size_t)l.bytes) return SS_EINVAL;

    const int expire = g_expire.exchange(-1, std::memory_order_relaxed);

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (grad && ss::linear_ce_fits_small(T, D, V)) return ss::linear_ce_small(a, st);
    unsigned char* ws = static_cast<unsigned char*>(a->workspace);
    Header* header = reinterpret_cast<Header*>(ws);
    int* row = reinterpret_cast<int*>(ws + l.row);
    int* target = reinterpret_cast<int*>(ws + l.target);
    float* target_logit = reinterpret_cast<float*>(ws + l.target_logit);
    float2* row_loss = reinterpret_cast<float2*>(ws + l.row_loss);
    double* partials = reinterpret_cast<double*>(ws + l.partials);
    uint16_t* h = reinterpret_cast<uint16_t*>(ws + l.h);
    int* counters = reinterpret_cast<int*>(ws + l.counters);
    const int mean = a->reduction == SS_LOSS_MEAN;

    GatherArgs ga = {header, a->targets, a->ignore_index, (int)T, (int)D, (int)l.Dp, (int)V,
                     static_cast<const uint16_t*>(a->hidden), a->hidden_stride, static_cast<const uint16_t*>(a->weight),
                     a->weight_stride, h, row, target, target_logit, a->token_loss_out,
                     static_cast<uint16_t*>(a->d_hidden), a->d_hidden_stride, (float)a->grad_scale, mean, counters,
                     (int)l.n_counters, nullptr};
    if (l.chunk) {
        int* chunk = reinterpret_cast<int*>(ws + l.chunk);
        if (int rc = ss::launch(ce_count_kernel, up(T, kChunk) / kChunk, kGatherThreads, 0, 0, true, st, a->targets,
                                a->ignore_index, T, chunk))
            return rc;
        ga.chunk = chunk;
    }
    if (!l.few)
        if (int rc = ss::launch(ce_gather_kernel, T > 0 ? (T + kGatherRows - 1) / kGatherRows : 1, kGatherThreads, 0, 0,
                                true, st, ga))
            return rc;

    const uint16_t* w = static_cast<const uint16_t*>(a->weight);
    int64_t ldw = a->weight_stride;
    if (stage) {
        uint16_t* staged = reinterpret_cast<uint16_t*>(ws + l.w);
        const int64_t per = kThreads / 32;
        if (int rc = ss::launch(ce_stage_kernel, (V + per - 1) / per, kThreads, 0, 0, true, st, w, ldw, V, D, l.Dp, l.few ? 1 : 0,
                                staged))
            return rc;
        w = staged;
        ldw = l.Dp;
    }

    GemmArgs g = {};
    g.header = header;
    g.next = counters;
    g.vocab = (int)V;
    g.log2e = (float)(kLog2eDouble * (1.0 + kDropped * (double)((std::min(D, kDroppedUpTo) + 15) / 16)));
    g.rows = (int)l.rows;
    g.target = target;
    g.token = row;
    g.row_loss = row_loss;
    g.loss = a->loss_out;
    g.stats = reinterpret_cast<float2*>(ws + l.stats);
    CUtensorMap h_k, w_k;
    const int64_t m_tiles = l.rows / kTile;
    if (T > 0) {
        if (int rc = make_map(&h_k, h, l.rows, D, l.Dp, kHalf)) return rc;
        if (int rc = make_map(&w_k, w, V, D, ldw, kHalf)) return rc;
        if (l.few) {
            const int rc = T == 1   ? launch_few<1>(ga, w, ldw, l.slices, l.rows, g.stats, st)
                           : T == 2 ? launch_few<2>(ga, w, ldw, l.slices, l.rows, g.stats, st)
                           : T == 3 ? launch_few<3>(ga, w, ldw, l.slices, l.rows, g.stats, st)
                                    : launch_few<kFewTokens>(ga, w, ldw, l.slices, l.rows, g.stats, st);
            if (rc) return rc;
        } else {
            Maps maps;
            maps.a[0] = h_k, maps.b[0] = w_k;
            Work& x = g.work[0];
            x.product = kStatistics;
            x.n_tiles = (int)l.n_tiles;
            x.splits = 1;
            x.k = (int)D;
            g.count = 1;
            g.expire = expire == 0;
            if (int rc = launch_gemm(maps, g, m_tiles * l.n_tiles, st)) return rc;
        }
    }
    const int64_t loss_blocks = T > 0 ? up(T, grad ? kBlockK : kLossRows) / kLossRows : 1;
    if (int rc = launch(ce_loss_kernel, loss_blocks, kLossThreads, 0, st, header, g.stats,
                        (int)l.slices, (int)l.rows, target_logit, row, row_loss, a->token_loss_out, partials, mean,
                        a->loss_out, grad && T > 0 ? h : nullptr, (int)l.Dp))
        return rc;
    if (!grad) return SS_OK;
    if (T == 0) {
        if (!a->d_weight) return SS_OK;
        const cudaError_t e =
            cudaMemset2DAsync(a->d_weight, (size_t)a->d_weight_stride * 2, 0, (size_t)D * 2, (size_t)V, st);
        return e == cudaSuccess ? SS_OK : ss::cuda_fail(e);
    }

    // Launch i: the gradients of piece i - 1 and the probabilities of piece i.
    uint16_t* p[2] = {reinterpret_cast<uint16_t*>(ws + l.p[0]), reinterpret_cast<uint16_t*>(ws + l.p[1])};
    CUtensorMap p_k[2], p_mn[2], h_mn, w_mn;
    for (int i = 0; i < 2; ++i) {
        if (int rc = make_map(&p_k[i], p[i], l.rows, l.piece, l.piece, kHalf)) return rc;
        if (int rc = make_map(&p_mn[i], p[i], l.rows, l.piece, l.piece, kBlockK)) return rc;
    }
    if (int rc = make_map(&h_mn, h, l.rows, D, l.Dp, kBlockK)) return rc;
    if (int rc = make_map(&w_mn, w, V, D, ldw, kBlockK)) return rc;
    const int64_t ld = up(D, 4), d_tiles = up(D, kTile) / kTile;
    for (int64_t i = 0; i <= l.pieces; ++i) {
        struct {
            Work work;
            const CUtensorMap *a, *b;
            int64_t tiles, blocks;
        } list[kMaxWork];
        int n = 0;
        const int64_t v0 = (i - 1) * l.piece;  // of the piece whose gradients are taken
        const int64_t rows_v = V - v0 < l.piece ? V - v0 : l.piece;
        const int64_t tiles_v = up(rows_v, kTile) / kTile;
        Work head = {};
        if (i > 0) {
            const int b = (int)((i - 1) & 1);
            if (a->d_hidden) {
                Work x = {};
                x.product = kHidden;
                x.n_tiles = (int)d_tiles;
                x.splits = l.hidden_splits;
                x.k = (int)(tiles_v * kTile);
                x.v0 = (int)v0;
                x.part = l.hidden_part ? reinterpret_cast<float*>(ws + l.hidden_part) : nullptr;
                x.part_split = l.rows * ld;
                x.part_ld = (int)ld;
                x.add = i > 1;
                x.out = static_cast<uint16_t*>(a->d_hidden);
                x.out_ld = a->d_hidden_stride;
                x.cols = (int)D;
                list[n++] = {x, &p_k[b], &w_mn, m_tiles * d_tiles * x.splits, tiles_v * kTile / kBlockK / x.splits};
            }
            if (a->d_weight) {
                head.product = kHead;
                head.m_tiles = (int)tiles_v;
                head.n_tiles = (int)d_tiles;
                head.splits = l.head_splits;
                head.v0 = (int)v0;
                head.part = l.head_part ? reinterpret_cast<float*>(ws + l.head_part) : nullptr;
                head.part_split = l.piece * ld;
                head.part_ld = (int)ld;
                head.out = static_cast<uint16_t*>(a->d_weight);
                head.out_ld = a->d_weight_stride;
                head.m_rows = (int)rows_v;
                head.cols = (int)D;
                list[n++] = {head, &p_mn[b], &h_mn, tiles_v * d_tiles * head.splits, l.rows / kBlockK / head.splits};
            }
        }
        if (i < l.pieces) {
            Work x = {};
            const int64_t left = l.n_tiles - i * (l.piece / kTile);
            x.product = kProbability;
            x.n_tiles = (int)(left < l.piece / kTile ? left : l.piece / kTile);
            x.splits = 1;
            x.k = (int)D;
            x.v0 = (int)(i * l.piece);
            x.p = p[i & 1];
            x.ldp = (int)l.piece;
            list[n++] = {x, &h_k, &w_k, m_tiles * x.n_tiles, up(D, kBlockK) / kBlockK};
        }
        std::stable_sort(list, list + n, [](const auto& x, const auto& y) { return x.blocks > y.blocks; });
        Maps maps;
        int64_t tiles = 0;
        for (int k = 0; k < n; ++k) {
            g.work[k] = list[k].work;
            maps.a[k] = *list[k].a, maps.b[k] = *list[k].b;
            tiles += list[k].tiles;
        }
        g.count = n;
        g.partials = i == 0 ? partials : nullptr;
        g.n_partials = (int)loss_blocks;
        g.mean = mean;
        g.expire = expire == i + 1;
        if (tiles > INT32_MAX - 1024) return SS_EOVERFLOW;
        if (int rc = launch_gemm(maps, g, tiles, st)) return rc;
        if (head.part) {
            const int64_t blocks = (rows_v * (ld / 4) + kThreads - 1) / kThreads;
            if (int rc = launch(ce_join_kernel, blocks, kThreads, 0, st, header, head.part, head.splits, head.part_split,
                                head.part_ld, (int)rows_v, (int)D, head.out + v0 * head.out_ld, head.out_ld, nullptr))
                return rc;
        }
    }
    if (a->d_hidden && l.hidden_part) {
        const int64_t blocks = (l.rows * (ld / 4) + kThreads - 1) / kThreads;
        return launch(ce_join_kernel, blocks, kThreads, 0, st, header, reinterpret_cast<float*>(ws + l.hidden_part),
                      l.hidden_splits, l.rows * ld, (int)ld, (int)l.rows, (int)D, static_cast<uint16_t*>(a->d_hidden),
                      a->d_hidden_stride, row);
    }
    return SS_OK;
}

}  // extern "C"
