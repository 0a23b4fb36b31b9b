// clip.cu -- the global gradient norm and clipping: over a list of tensors,
// and over the reduced gradients of a sharded plan with AdamW on what is
// clipped.
//
//   n = sqrt(sum over every element of x^2),  c = min(1, max_norm / (n + 1e-6)),
//   x <- c * x
// (c is NaN where n is; n is +inf once a square passes fp32, from |x| = 1.8e19
// on, and c is then 0; a max_norm of +inf never clips, whatever n is).  Nothing can be scaled before everything has been
// read, so the work is two passes over the data with the factor between them:
//
//   pass 1  each CTA squares and sums its part of the elements in fp32 (at most
//           32 values a thread, then the 256 threads) and writes one partial;
//   fold    the partials are summed in fp64 in one fixed order, so the norm
//           does not depend on which CTA ran first;
//   pass 2  every element is scaled by the factor.
//
// A list small enough for one cluster of CTAs takes a single launch: the data stay
// in registers between the passes, and the CTAs' sums meet in one another's
// shared memory.
//
// All of it is bound by HBM (2 flops per 2 bytes read), or, where there is
// little of it, by launches.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "adamw.cuh"
#include "device_utils.cuh"
#include "internal.h"
#include "launch.cuh"
#include "segmap.cuh"

namespace {

using ss::AdamCoef;

constexpr int kThreads = 256;
constexpr int kVecs = 4;                         // 16-byte blocks per thread of a tile
constexpr int kTileBlocks = kThreads * kVecs;    // 16 KiB: a tile is one of these, or more (list_rounds)
constexpr int kTab = 512;                        // tensors per launch
constexpr int kTabSmall = 16;                    // of the one-cluster form (a short parameter block)
constexpr double kEps = 1e-6;                    // added to the norm in the factor's denominator
constexpr double kNormOnly = -INFINITY;          // max_norm of a call that scales nothing: its factor is 1
constexpr int kFoldSpan = 8192;                  // partials summed by one CTA of the first fold

// The workspace: fp32 partials, then the doubles of a first fold.
constexpr int64_t kMaxPartials = SS_NORM_WORKSPACE_BYTES / 4 - 2 * 1024;
constexpr int64_t kMaxFold = 1024;
static_assert(kMaxPartials / kFoldSpan < kMaxFold, "the first fold's doubles fit the workspace");
static_assert((kMaxPartials * 4) % 16 == 0, "the first fold's doubles are aligned");

// The tensors of one launch: start, first tile and element count of each
// (elements are negated for fp32).
template <int S>
struct ListTabT {
    const unsigned char* in[S];
    unsigned char* out[S];
    int64_t n[S];
    int first[S + 1];
    int count;
};
using ListTab = ListTabT<kTab>;

struct RankPtrs {
    const void* p[SS_MAX_WORLD];
};

// The tensor of a tile: the last one whose first tile is at or before it.
__device__ __forceinline__ int find_tensor(const int* first, int count, int tile) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float square_sum_bf16(uint4 w, float s) {
    float x;
    x = ss::bf16_lo(w.x); s = fmaf(x, x, s);
    x = ss::bf16_hi(w.x); s = fmaf(x, x, s);
    x = ss::bf16_lo(w.y); s = fmaf(x, x, s);
    x = ss::bf16_hi(w.y); s = fmaf(x, x, s);
    x = ss::bf16_lo(w.z); s = fmaf(x, x, s);
    x = ss::bf16_hi(w.z); s = fmaf(x, x, s);
    x = ss::bf16_lo(w.w); s = fmaf(x, x, s);
    x = ss::bf16_hi(w.w); s = fmaf(x, x, s);
    return s;
}

__device__ __forceinline__ float square_sum_f32(uint4 w, float s) {
    float x;
    x = __uint_as_float(w.x); s = fmaf(x, x, s);
    x = __uint_as_float(w.y); s = fmaf(x, x, s);
    x = __uint_as_float(w.z); s = fmaf(x, x, s);
    x = __uint_as_float(w.w); s = fmaf(x, x, s);
    return s;
}

// w with the bytes outside [lo, hi) zeroed (lo, hi multiples of 2).
__device__ __forceinline__ uint4 keep_bytes(uint4 w, int lo, int hi) {
    uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int b = 0; b < 16; b += 2)
        if (b < lo || b >= hi) v[b >> 2] &= (b & 2) ? 0x0000FFFFu : 0xFFFF0000u;
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// Sum over the CTA of kThreads threads, in a fixed order; valid in thread 0.
template <class T>
__device__ __forceinline__ T block_sum(T s) {
    __shared__ T part[kThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_down_sync(0xFFFFFFFFu, s, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = threadIdx.x < kThreads / 32 ? part[threadIdx.x] : T(0);
#pragma unroll
        for (int d = kThreads / 64; d > 0; d >>= 1) s += __shfl_down_sync(0xFFFFFFFFu, s, d);
    }
    return s;
}

// Pass 1 over a list: one tile of aligned 16-byte blocks of one tensor.  300 M bf16
// elements in 85 us: 7.04 TB/s, 89 % of the DRAM's rate.  The
// blocks at a tensor's ends may hold bytes of something else; they lie in the
// same 16 bytes as one of its own, and are masked out.
__global__ void __launch_bounds__(kThreads)
list_square_kernel(const __grid_constant__ ListTab tab, int rounds, float* __restrict__ partials) {
    ss::launch_after();
    const int tile = blockIdx.x;
    const int k = find_tensor(tab.first, tab.count, tile);
    ss::wait_before();
    const unsigned char* p = tab.in[k];
    const int64_t n = tab.n[k];
    const int64_t bytes = n < 0 ? -n * 4 : n * 2;
    const int lead = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
    const int64_t end = lead + bytes;  // of the tensor, from the first block's start
    const unsigned char* base = p - lead;
    int64_t b0 = (int64_t)(tile - tab.first[k]) * rounds * kTileBlocks + threadIdx.x;
    float s = 0.f;
    for (int it = 0; it < rounds; ++it, b0 += kTileBlocks) {
        uint4 w[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t at = 16 * (b0 + i * kThreads);
            w[i] = make_uint4(0, 0, 0, 0);
            if (at < end) w[i] = ss::ld_stream_u4(base + at);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t at = 16 * (b0 + i * kThreads);
            if (at < lead || at + 16 > end) {
                const int lo = at < lead ? lead : 0;
                const int hi = end - at < 16 ? (end - at > 0 ? (int)(end - at) : 0) : 16;
                w[i] = keep_bytes(w[i], lo, hi);
            }
            s = n < 0 ? square_sum_f32(w[i], s) : square_sum_bf16(w[i], s);
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) partials[tile] = s;
}

// First fold, for many partials: CTA b sums partials [b * kFoldSpan, ...).
__global__ void __launch_bounds__(kThreads)
fold_kernel(const float* __restrict__ partials, int64_t n, double* __restrict__ sums) {
    ss::launch_after();
    ss::wait_before();
    const int64_t a = (int64_t)blockIdx.x * kFoldSpan;
    const int64_t b = a + kFoldSpan < n ? a + kFoldSpan : n;
    double s = 0.0;
    for (int64_t i = a + threadIdx.x; i < b; i += kThreads) s += (double)partials[i];
    s = block_sum(s);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// The norm and the factor of a sum of squares, in fp32 where the sum is in its
// range (fp64 roots and quotients take hundreds of clocks).  A NaN norm gives a
// NaN factor (min would drop it); an infinite one is not divided into an infinite
// max_norm.
__device__ __forceinline__ void write_norm(double sq, double max_norm, float* norm_out) {
    float norm, c;
    if (sq > 1e-30 && sq < 1e38) {
        norm = __fsqrt_rn((float)sq);
        c = __fdiv_rn(fabsf((float)max_norm), norm + (float)kEps);
    } else {
        const double n = sqrt(sq);
        norm = (float)n;
        if (isinf(max_norm))
            c = max_norm > 0.0 && isnan(norm) ? norm : 1.0f;
        else
            c = (float)(max_norm / (n + kEps));
    }
    norm_out[0] = norm;
    norm_out[1] = c >= 1.0f ? 1.0f : c;
}

// Last fold, one CTA: the sum of n partials, as it is (sq_out) or as norm and
// factor (norm_out); either may be NULL.
template <class T>
__global__ void __launch_bounds__(kThreads)
finish_kernel(const T* v, int64_t n, double max_norm, double* sq_out, float* norm_out) {
    ss::launch_after();
    ss::wait_before();
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += (double)v[i];
    s = block_sum(s);
    if (threadIdx.x == 0) {
        if (sq_out) *sq_out = s;
        if (norm_out) write_norm(s, max_norm, norm_out);
    }
}

// Sum of n doubles by one warp, the same in every lane and whichever kernel asks.
__device__ __forceinline__ double sum_sums(const double* sq, int n) {
    double s = 0.0;
    for (int i = threadIdx.x & 31; i < n; i += 32) s += sq[i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    return s;
}

// Norm and factor of the sums of a sharded step; one warp.  Its successor may
// start when this one's own predecessors are done, and has the factor to wait for.
__global__ void norm_kernel(const double* sq, int n, double max_norm, float* norm_out) {
    ss::wait_before();
    ss::launch_after();
    const double s = sum_sums(sq, n);
    if (threadIdx.x == 0) write_norm(s, max_norm, norm_out);
}

__device__ __forceinline__ uint4 scale_bf16(uint4 w, float c) {
    return make_uint4(ss::pack_bf16x2(ss::bf16_lo(w.x) * c, ss::bf16_hi(w.x) * c),
                      ss::pack_bf16x2(ss::bf16_lo(w.y) * c, ss::bf16_hi(w.y) * c),
                      ss::pack_bf16x2(ss::bf16_lo(w.z) * c, ss::bf16_hi(w.z) * c),
                      ss::pack_bf16x2(ss::bf16_lo(w.w) * c, ss::bf16_hi(w.w) * c));
}

__device__ __forceinline__ uint4 scale_f32(uint4 w, float c) {
    return make_uint4(__float_as_uint(__uint_as_float(w.x) * c), __float_as_uint(__uint_as_float(w.y) * c),
                      __float_as_uint(__uint_as_float(w.z) * c), __float_as_uint(__uint_as_float(w.w) * c));
}

// 16 bytes this kernel may also write (not .nc).
__device__ __forceinline__ uint4 ld_rw_u4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Pass 2 over a list, 300 M bf16 elements in 167 us (7.2 TB/s with what is in L2
// still): one tile of a tensor's output, in aligned 16-byte blocks
// of the output; an input at another offset is realigned in registers, and the
// blocks at the tensor's ends go element by element.  In place with a factor of
// 1 there is nothing to write.  SELF: every CTA folds the (few) partials itself,
// the first one writes the result down.
template <bool SELF>
__global__ void __launch_bounds__(kThreads)
list_scale_kernel(const __grid_constant__ ListTab tab, int rounds, const float* partials, int n_partials,
                  double max_norm, float* norm) {
    ss::launch_after();
    ss::wait_before();
    float c;
    if (SELF) {
        __shared__ float result[2];
        double sum = 0.0;
        for (int i = threadIdx.x; i < n_partials; i += kThreads) sum += (double)partials[i];
        sum = block_sum(sum);
        if (threadIdx.x == 0) {
            write_norm(sum, max_norm, result);
            if (blockIdx.x == 0) norm[0] = result[0], norm[1] = result[1];
        }
        __syncthreads();
        c = result[1];
    } else {
        c = norm[1];
    }
    const int tile = gridDim.x - 1 - blockIdx.x;  // what pass 1 read last is in L2 still
    const int k = find_tensor(tab.first, tab.count, tile);
    const unsigned char* in = tab.in[k];
    unsigned char* out = tab.out[k];
    if (c == 1.0f && in == out) return;
    const int64_t n = tab.n[k];
    const int eb = n < 0 ? 4 : 2;
    const int64_t bytes = n < 0 ? -n * 4 : n * 2;
    const int lead = (int)(reinterpret_cast<uintptr_t>(out) & 15u);
    const bool congruent = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    int64_t b0 = (int64_t)(tile - tab.first[k]) * rounds * kTileBlocks + threadIdx.x;
    for (int it = 0; it < rounds; ++it, b0 += kTileBlocks) {
        uint4 w[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t at = 16 * (b0 + i * kThreads) - lead;  // byte offset inside the tensor
            if (at >= 0 && at + 16 <= bytes) w[i] = congruent ? ld_rw_u4(in + at) : ss::ld_any16(in + at);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t at = 16 * (b0 + i * kThreads) - lead;
            if (at >= 0 && at + 16 <= bytes) {
                ss::st_stream_u4(out + at, eb == 4 ? scale_f32(w[i], c) : scale_bf16(w[i], c));
            } else {
                for (int64_t x = at < 0 ? 0 : at; x < at + 16 && x < bytes; x += eb) {
                    if (eb == 4)
                        *reinterpret_cast<float*>(out + x) = *reinterpret_cast<const float*>(in + x) * c;
                    else
                        *reinterpret_cast<uint16_t*>(out + x) =
                            ss::f32_to_bf16(ss::bf16_to_f32(*reinterpret_cast<const uint16_t*>(in + x)) * c);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// a list in one cluster
// ---------------------------------------------------------------------------

constexpr int kClusterMax = 8;                          // the portable size
constexpr int kSmallRounds = 2;                         // 4 KiB tiles of a CTA, held in registers
constexpr int kSmallTiles = kClusterMax * kSmallRounds;
constexpr int kTabMid = 256;                            // tensors of the cooperative form
constexpr int kMidCtas = 4;                             // its CTAs an SM
constexpr int kMidRounds = 4;                           // tiles of each: 10 MB on 152 SMs

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Sum over a cluster of one fp32 value per CTA (thread 0's), in rank order and
// in fp64, the same in every thread of every CTA.  All threads take part, and
// call cluster_wait() before they leave: their CTA's value may still be read.
__device__ __forceinline__ double cluster_sum(float s) {
    __shared__ float mine;
    if (threadIdx.x == 0) mine = s;
    cluster_arrive();
    cluster_wait();
    const int n = (int)cluster_size(), lane = threadIdx.x & 31;
    float x = 0.f;
    if (lane < n) {
        uint32_t at = (uint32_t)__cvta_generic_to_shared(&mine);
        asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(lane));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    }
    __syncwarp();
    cluster_arrive();
    double sum = 0.0;
    for (int i = 0; i < n; ++i) sum += (double)__shfl_sync(0xFFFFFFFFu, x, i);
    return sum;
}

// Tiles `first`, first + step, ... of a list (256 aligned 16-byte blocks of the
// outputs each) held in registers, one block a thread; every load goes out before
// the first square.
template <int ROUNDS>
struct Held {
    uint4 w[ROUNDS];
    int k[ROUNDS];  // tensor, -1 for no tile

    template <class Tab>
    __device__ __forceinline__ void load(const Tab& tab, int first, int step) {
        const int tiles = tab.first[tab.count];
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            const int tile = first + i * step;
            w[i] = make_uint4(0, 0, 0, 0);
            k[i] = -1;
            if (tile >= tiles) continue;
            k[i] = find_tensor(tab.first, tab.count, tile);
            const unsigned char* in = tab.in[k[i]];
            const int64_t n = tab.n[k[i]], bytes = n < 0 ? -n * 4 : n * 2;
            const int64_t at = offset(tab, tile, k[i]);
            if (at >= 0 && at + 16 <= bytes) {
                w[i] = (reinterpret_cast<uintptr_t>(in + at) & 15u) == 0 ? ld_rw_u4(in + at) : ss::ld_any16(in + at);
            } else if (at < bytes) {
                uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
                for (int b = 0; b < 16; b += 2)
                    if (at + b >= 0 && at + b < bytes)
                        v[b >> 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(in + at + b) << (8 * (b & 2));
                w[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    }

    // byte offset of this thread's block in tensor k
    template <class Tab>
    __device__ __forceinline__ int64_t offset(const Tab& tab, int tile, int k) const {
        const int lead = (int)(reinterpret_cast<uintptr_t>(tab.out[k]) & 15u);
        return 16 * ((int64_t)(tile - tab.first[k]) * kThreads + threadIdx.x) - lead;
    }

    template <class Tab>
    __device__ __forceinline__ float square_sum(const Tab& tab) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i)
            if (k[i] >= 0) s = tab.n[k[i]] < 0 ? square_sum_f32(w[i], s) : square_sum_bf16(w[i], s);
        return s;
    }

    template <class Tab>
    __device__ __forceinline__ void store_scaled(const Tab& tab, int first, int step, float c) const {
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            if (k[i] < 0) continue;
            unsigned char* out = tab.out[k[i]];
            if (c == 1.0f && tab.in[k[i]] == out) continue;
            const int64_t n = tab.n[k[i]], bytes = n < 0 ? -n * 4 : n * 2;
            const int64_t at = offset(tab, first + i * step, k[i]);
            const uint4 v = n < 0 ? scale_f32(w[i], c) : scale_bf16(w[i], c);
            if (at >= 0 && at + 16 <= bytes)
                *reinterpret_cast<uint4*>(out + at) = v;
            else if (at < bytes)
                ss::st_bytes(out + at, v, at < 0 ? (int)-at : 0, bytes - at < 16 ? (int)(bytes - at) : 16);
        }
    }
};

// Norm, and (scale) clipping, of a list in one launch: one cluster.
__global__ void __launch_bounds__(kThreads)
list_small_kernel(const __grid_constant__ ListTabT<kTabSmall> tab, double max_norm, int scale, float* norm_out) {
    ss::launch_after();
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    Held<kSmallRounds> held;
    ss::wait_before();
    held.load(tab, rank, ranks);
    const double sq = cluster_sum(block_sum(held.square_sum(tab)));
    float result[2];
    write_norm(sq, max_norm, result);
    if (threadIdx.x == 0 && rank == 0) norm_out[0] = result[0], norm_out[1] = result[1];
    if (scale) held.store_scaled(tab, rank, ranks, result[1]);
    __syncwarp();
    cluster_wait();
}

// The same on the whole GPU: a cooperative launch, whose CTAs (all resident at
// once) meet between the passes at the grid's barrier.  Every CTA sums all the
// partials, in one order.  200 odd tensors, 1.3 MB: 8.8 us a call, 9.8 by two
// launches; one of 750 KB: 6.6, 8.2.
__global__ void __launch_bounds__(kThreads, kMidCtas)
list_mid_kernel(const __grid_constant__ ListTabT<kTabMid> tab, double max_norm, int scale, float* partials,
                float* norm_out) {
    const int rank = blockIdx.x, ranks = gridDim.x;
    Held<kMidRounds> held;
    held.load(tab, rank, ranks);
    const float s = block_sum(held.square_sum(tab));
    if (threadIdx.x == 0) partials[rank] = s;
    cooperative_groups::this_grid().sync();
    double sum = 0.0;
    for (int i = threadIdx.x; i < ranks; i += kThreads) sum += (double)__ldcg(partials + i);
    sum = block_sum(sum);
    __shared__ float result[2];
    if (threadIdx.x == 0) {
        write_norm(sum, max_norm, result);
        if (rank == 0) norm_out[0] = result[0], norm_out[1] = result[1];
    }
    if (!scale) return;
    __syncthreads();
    held.store_scaled(tab, rank, ranks, result[1]);
}

// ---------------------------------------------------------------------------
// the sharded form
// ---------------------------------------------------------------------------

// 16 bytes of plan elements as fp32 values (8 bf16 or 4 fp32).
template <int EB>
struct Vec {
    static constexpr int n = 16 / EB;
};

template <int EB>
__device__ __forceinline__ void widen(uint4 w, float (&x)[16 / EB]) {
    if constexpr (EB == 2) {
        x[0] = ss::bf16_lo(w.x); x[1] = ss::bf16_hi(w.x); x[2] = ss::bf16_lo(w.y); x[3] = ss::bf16_hi(w.y);
        x[4] = ss::bf16_lo(w.z); x[5] = ss::bf16_hi(w.z); x[6] = ss::bf16_lo(w.w); x[7] = ss::bf16_hi(w.w);
    } else {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
}

// A plan range as whole vectors and the elements left at its two ends (fewer
// than 16 in all), which one CTA's first warp takes one by one.
struct Split {
    int64_t vbeg, nvec, a0, a1, b0, b1;
    // the element of an edge thread, -1 for none
    __device__ __forceinline__ int64_t edge(int t) const {
        return t < a1 - a0 ? a0 + t : t - (a1 - a0) < b1 - b0 ? b0 + (t - (a1 - a0)) : -1;
    }
};

// Reduce-scatter of one vector per thread and round: g = (G_0 + ... + G_{N-1}) / N
// in rank order, written, and the CTA's sum of g^2 as one partial; CLUSTER: the
// whole grid is one cluster, which sums the partials itself.  Pads hold zero
// gradients and add nothing.  CTA b takes `rounds` consecutive rounds of kThreads
// vectors (one, unless the partials would not fit).  Short CTAs in address order, as
// in the unclipped step: 50 M bf16 parameters of 7 ranks in 124 us, 7.3 TB/s.
template <int NR, int EB, bool CLUSTER>
__global__ void __launch_bounds__(kThreads)
rs_square_kernel(RankPtrs grads, int N, Split sp, int rounds, float* __restrict__ gout,
                 float* __restrict__ partials, double* __restrict__ sq_out) {
    ss::launch_after();
    ss::wait_before();
    constexpr int E = Vec<EB>::n;
    const int n = NR > 0 ? NR : N;
    const float fN = (float)n;
    float sq = 0.f;
    for (int it = 0; it < rounds; ++it) {
        const int64_t q = ((int64_t)blockIdx.x * rounds + it) * kThreads + threadIdx.x;
        if (q >= sp.nvec) break;
        const int64_t at = (sp.vbeg + q * E) * EB;  // byte offset of the vector
        constexpr int kW = NR > 0 ? NR : 8;
        uint4 w[kW];
#pragma unroll
        for (int r = 0; r < kW; ++r)
            if (NR > 0 || r < n) w[r] = ss::ld_stream_u4(static_cast<const unsigned char*>(grads.p[r]) + at);
        float s[E], x[E];
        widen<EB>(w[0], s);
#pragma unroll
        for (int r = 1; r < kW; ++r) {
            if (NR > 0 || r < n) {
                widen<EB>(w[r], x);
#pragma unroll
                for (int e = 0; e < E; ++e) s[e] = __fadd_rn(s[e], x[e]);
            }
        }
        // ranks beyond the first 8 (N > 8), 8 loads in flight at a time
        for (int r0 = 8; NR == 0 && r0 < n; r0 += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (r0 + j < n)
                    w[j] = ss::ld_stream_u4(static_cast<const unsigned char*>(grads.p[r0 + j]) + at);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (r0 + j < n) {
                    widen<EB>(w[j], x);
#pragma unroll
                    for (int e = 0; e < E; ++e) s[e] = __fadd_rn(s[e], x[e]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[e] = __fdiv_rn(s[e], fN);
            sq = fmaf(s[e], s[e], sq);
        }
        float* o = gout + sp.vbeg + q * E;
#pragma unroll
        for (int e = 0; e < E; e += 4) ss::st_stream_f4(o + e, make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]));
    }
    const int64_t f = blockIdx.x == gridDim.x - 1 ? sp.edge(threadIdx.x) : -1;
    if (f >= 0) {
        float s = 0.f;
        for (int r = 0; r < n; ++r) {
            const float x = EB == 2 ? ss::bf16_to_f32(static_cast<const uint16_t*>(grads.p[r])[f])
                                    : static_cast<const float*>(grads.p[r])[f];
            s = r == 0 ? x : __fadd_rn(s, x);
        }
        s = __fdiv_rn(s, fN);
        gout[f] = s;
        sq = fmaf(s, s, sq);
    }
    sq = block_sum(sq);
    if (CLUSTER) {
        const double sum = cluster_sum(sq);
        if (threadIdx.x == 0 && blockIdx.x == 0) *sq_out = sum;
        __syncwarp();
        cluster_wait();
    } else if (threadIdx.x == 0) {
        partials[blockIdx.x] = sq;
    }
}

// AdamW on the clipped reduced gradient, one vector of plan elements per
// thread.  MASTER == false: theta is the shard itself (no fp32 master).  SELF:
// every CTA works the factor out of the sums (CTA 0 writes it down), else
// norm_kernel has done it.  The state is on its way before the factor is known.
// 50 M bf16 parameters in 220 us: 6.8 TB/s.
template <int EB, bool MASTER, bool SELF>
__global__ void __launch_bounds__(kThreads)
clip_adamw_kernel(const float* __restrict__ reduced, const double* sq, int num_sums, double max_norm, float* norm,
                  Split sp, float* __restrict__ master, float* __restrict__ exp_avg,
                  float* __restrict__ exp_avg_sq, unsigned char* __restrict__ shards, AdamCoef c) {
    if (SELF) {
        ss::launch_after();
        ss::wait_before();
    }
    constexpr int E = Vec<EB>::n;
    const int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t f = sp.vbeg + q * E;
    const bool whole = q < sp.nvec;
    float4 g[E / 4], t[E / 4], m[E / 4], v[E / 4];
    if (whole) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const uint4 w = ss::ld_stream_u4(reduced + f + 4 * i);
            g[i] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
            if (MASTER) t[i] = ss::ld_rw_f4(master + f + 4 * i);
            m[i] = ss::ld_rw_f4(exp_avg + f + 4 * i);
            v[i] = ss::ld_rw_f4(exp_avg_sq + f + 4 * i);
        }
        if (!MASTER) {
            float x[E];
            widen<EB>(ld_rw_u4(shards + f * EB), x);
#pragma unroll
            for (int i = 0; i < E / 4; ++i) t[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
    }
    float clip;
    if (SELF) {
        __shared__ float result[2];
        if (threadIdx.x < 32) {
            const double s = sum_sums(sq, num_sums);
            if (threadIdx.x == 0) {
                write_norm(s, max_norm, result);
                if (blockIdx.x == 0) norm[0] = result[0], norm[1] = result[1];
            }
        }
        __syncthreads();
        clip = result[1];
    } else {
        ss::wait_before();
        clip = norm[1];
    }
    if (whole) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            ss::adamw_elem(__fmul_rn(g[i].x, clip), t[i].x, m[i].x, v[i].x, c);
            ss::adamw_elem(__fmul_rn(g[i].y, clip), t[i].y, m[i].y, v[i].y, c);
            ss::adamw_elem(__fmul_rn(g[i].z, clip), t[i].z, m[i].z, v[i].z, c);
            ss::adamw_elem(__fmul_rn(g[i].w, clip), t[i].w, m[i].w, v[i].w, c);
            if (MASTER) ss::st_stream_f4(master + f + 4 * i, t[i]);
            ss::st_stream_f4(exp_avg + f + 4 * i, m[i]);
            ss::st_stream_f4(exp_avg_sq + f + 4 * i, v[i]);
        }
        uint4 p;
        if constexpr (EB == 2) {
            p = make_uint4(ss::pack_bf16x2(t[0].x, t[0].y), ss::pack_bf16x2(t[0].z, t[0].w),
                           ss::pack_bf16x2(t[1].x, t[1].y), ss::pack_bf16x2(t[1].z, t[1].w));
        } else {
            p = make_uint4(__float_as_uint(t[0].x), __float_as_uint(t[0].y), __float_as_uint(t[0].z),
                           __float_as_uint(t[0].w));
        }
        ss::st_stream_u4(shards + f * EB, p);
    }
    const int64_t x = blockIdx.x == gridDim.x - 1 ? sp.edge(threadIdx.x) : -1;
    if (x >= 0) {
        uint16_t* s16 = reinterpret_cast<uint16_t*>(shards);
        float* s32 = reinterpret_cast<float*>(shards);
        float th = MASTER ? master[x] : EB == 2 ? ss::bf16_to_f32(s16[x]) : s32[x];
        float m1 = exp_avg[x], v1 = exp_avg_sq[x];
        ss::adamw_elem(__fmul_rn(reduced[x], clip), th, m1, v1, c);
        if (MASTER) master[x] = th;
        exp_avg[x] = m1;
        exp_avg_sq[x] = v1;
        if (EB == 2)
            s16[x] = ss::f32_to_bf16(th);
        else
            s32[x] = th;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

Split split_range(int64_t lo, int64_t hi, int e) {
    Split s;
    s.vbeg = (lo + e - 1) / e * e;
    const int64_t vend = hi / e * e;
    if (vend > s.vbeg) {
        s.nvec = (vend - s.vbeg) / e;
        s.a0 = lo, s.a1 = s.vbeg, s.b0 = vend, s.b1 = hi;
    } else {
        s.nvec = 0;
        s.a0 = lo, s.a1 = hi, s.b0 = s.b1 = hi;
    }
    return s;
}

// n fp32 partials at the workspace's start to one sum, norm and factor.
int fold(void* workspace, int64_t n, double max_norm, double* sq_out, float* norm_out, cudaStream_t st) {
    float* partials = static_cast<float*>(workspace);
    if (n <= kFoldSpan)
        return ss::launch(finish_kernel<float>, 1, kThreads, 0, 0, true, st, partials, n, max_norm, sq_out, norm_out);
    double* sums = reinterpret_cast<double*>(partials + kMaxPartials);
    const int64_t blocks = (n + kFoldSpan - 1) / kFoldSpan;
    if (int rc = ss::launch(fold_kernel, blocks, kThreads, 0, 0, true, st, partials, n, sums)) return rc;
    return ss::launch(finish_kernel<double>, 1, kThreads, 0, 0, true, st, sums, blocks, max_norm, sq_out, norm_out);
}

int check_workspace(const void* workspace, size_t bytes) {
    if (!workspace || bytes < SS_NORM_WORKSPACE_BYTES) return SS_EINVAL;
    return ss::aligned(workspace, 16) ? SS_OK : SS_EALIGN;
}

int64_t tiles_of(const void* p, int64_t bytes, int rounds) {
    const int64_t blocks = ((int64_t)(reinterpret_cast<uintptr_t>(p) & 15u) + bytes + 15) / 16;
    const int64_t per = (int64_t)kTileBlocks * rounds;
    return (blocks + per - 1) / per;
}

int check_list(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads,
               const void* const* out) {
    if (num_tensors < 0 || (num_tensors > 0 && (!numels || !elem_bytes || !grads))) return SS_EINVAL;
    int64_t all = 0;  // bytes of all tensors
    for (int k = 0; k < num_tensors; ++k) {
        const int eb = elem_bytes[k];
        if (numels[k] < 0 || (eb != 2 && eb != 4)) return SS_EINVAL;
        if (numels[k] > (INT64_MAX >> 8) / eb || all > (INT64_MAX >> 8)) return SS_EOVERFLOW;
        all += numels[k] * eb;
        if (numels[k] == 0) continue;
        if (!grads[k] || (out && !out[k])) return SS_EINVAL;
        if (!ss::aligned(grads[k], eb) || (out && !ss::aligned(out[k], eb))) return SS_EALIGN;
    }
    return SS_OK;
}

// 16 KiB rounds in a tile: 1, unless the list has so many tiles that their
// partials would not fit the workspace (above 16 GB).  0: not even then.
int list_rounds(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads) {
    for (int64_t rounds = 1; rounds <= (1 << 20); rounds *= 2) {
        int64_t tiles = 0;
        for (int k = 0; k < num_tensors; ++k)
            if (numels[k] > 0) tiles += tiles_of(grads[k], numels[k] * elem_bytes[k], (int)rounds);
        if (tiles <= kMaxPartials) return (int)rounds;
    }
    return 0;
}

// Runs `launch` over the non-empty tensors, kTab at a time, tiled by the
// alignment of the inputs or (by_out) of the outputs.
template <class Launch>
int for_tables(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads,
               void* const* out, bool by_out, int rounds, Launch launch) {
    ListTab tab;
    tab.count = 0;
    tab.first[0] = 0;
    for (int k = 0; k < num_tensors; ++k) {
        if (numels[k] > 0) {
            const int j = tab.count++;
            tab.in[j] = static_cast<const unsigned char*>(grads[k]);
            tab.out[j] = static_cast<unsigned char*>(out ? out[k] : const_cast<void*>(grads[k]));
            tab.n[j] = elem_bytes[k] == 4 ? -numels[k] : numels[k];
            const void* by = by_out ? tab.out[j] : tab.in[j];
            tab.first[j + 1] = tab.first[j] + (int)tiles_of(by, numels[k] * elem_bytes[k], rounds);
        }
        if (tab.count > 0 && (tab.count == kTab || k == num_tensors - 1)) {
            if (int rc = launch(tab)) return rc;
            tab.count = 0;
        }
    }
    return SS_OK;
}

int cluster_for(int64_t ctas) {
    int c = 1;
    while (c < kClusterMax && c < ctas) c *= 2;
    return c;
}

// The whole call in one launch, where the list fits a cluster: kNotSmall if not.
constexpr int kNotSmall = 1;

template <int S>
int fill_table(ListTabT<S>& tab, int64_t max_tiles, int num_tensors, const int64_t* numels, const int* elem_bytes,
               const void* const* grads, void* const* out) {
    tab.count = 0;
    tab.first[0] = 0;
    for (int k = 0; k < num_tensors; ++k) {
        if (numels[k] == 0) continue;
        if (tab.count == S) return kNotSmall;
        const int j = tab.count;
        tab.in[j] = static_cast<const unsigned char*>(grads[k]);
        tab.out[j] = static_cast<unsigned char*>(out ? out[k] : const_cast<void*>(grads[k]));
        tab.n[j] = elem_bytes[k] == 4 ? -numels[k] : numels[k];
        const int64_t blocks =
            ((int64_t)(reinterpret_cast<uintptr_t>(tab.out[j]) & 15u) + numels[k] * elem_bytes[k] + 15) / 16;
        const int64_t tiles = tab.first[j] + (blocks + kThreads - 1) / kThreads;
        if (tiles > max_tiles) return kNotSmall;
        tab.first[j + 1] = (int)tiles;
        tab.count = j + 1;
    }
    return SS_OK;
}

int list_small(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads,
               void* const* out, bool scale, double max_norm, float* norm_out, cudaStream_t st) {
    ListTabT<kTabSmall> tab;
    if (int rc = fill_table(tab, kSmallTiles, num_tensors, numels, elem_bytes, grads, out)) return rc;
    const int cluster = cluster_for(tab.first[tab.count]);
    return ss::launch(list_small_kernel, cluster, kThreads, 0, cluster, true, st, tab, max_norm, scale ? 1 : 0, norm_out);
}

int list_mid(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads,
             void* const* out, bool scale, double max_norm, float* norm_out, float* partials, cudaStream_t st) {
    ListTabT<kTabMid> tab;
    const int64_t most = (int64_t)ss::num_sms() * kMidCtas;
    if (int rc = fill_table(tab, most * kMidRounds, num_tensors, numels, elem_bytes, grads, out)) return rc;
    const int64_t tiles = tab.first[tab.count];
    const int rc = ss::launch_cooperative(list_mid_kernel, tiles < most ? tiles : most, kThreads, st, tab, max_norm,
                                          scale ? 1 : 0, partials, norm_out);
    return rc == ss::kNotResident ? kNotSmall : rc;
}

// Partials up to which the second pass folds them itself, in every CTA.
constexpr int64_t kSelfPartials = 1024;

int list_call(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads,
              void* const* out, bool scale, double max_norm, float* norm_out, void* workspace, cudaStream_t st) {
    int rc = list_small(num_tensors, numels, elem_bytes, grads, out, scale, max_norm, norm_out, st);
    if (rc != kNotSmall) return rc;
    rc = list_mid(num_tensors, numels, elem_bytes, grads, out, scale, max_norm, norm_out, static_cast<float*>(workspace),
                  st);
    if (rc != kNotSmall) return rc;
    const int rounds = list_rounds(num_tensors, numels, elem_bytes, grads);
    if (rounds == 0) return SS_EOVERFLOW;
    float* partials = static_cast<float*>(workspace);
    int64_t n = 0;
    rc = for_tables(num_tensors, numels, elem_bytes, grads, nullptr, false, rounds, [&](const ListTab& tab) {
        const int tiles = tab.first[tab.count];
        const int rc1 = ss::launch(list_square_kernel, tiles, kThreads, 0, 0, true, st, tab, rounds, partials + n);
        n += tiles;
        return rc1;
    });
    if (rc) return rc;
    const bool self = scale && n <= kSelfPartials;
    if (!self)
        if ((rc = fold(workspace, n, max_norm, nullptr, norm_out, st))) return rc;
    if (!scale) return SS_OK;
    return for_tables(num_tensors, numels, elem_bytes, grads, out, true, rounds, [&](const ListTab& tab) {
        return ss::launch(self ? list_scale_kernel<true> : list_scale_kernel<false>, tab.first[tab.count], kThreads, 0, 0,
                          true, st, tab, rounds, partials, (int)n, max_norm, norm_out);
    });
}

template <int EB, bool CLUSTER>
auto pick_square(int N) {
    switch (N) {
        case 1: return rs_square_kernel<1, EB, CLUSTER>;
        case 2: return rs_square_kernel<2, EB, CLUSTER>;
        case 3: return rs_square_kernel<3, EB, CLUSTER>;
        case 4: return rs_square_kernel<4, EB, CLUSTER>;
        case 5: return rs_square_kernel<5, EB, CLUSTER>;
        case 6: return rs_square_kernel<6, EB, CLUSTER>;
        case 7: return rs_square_kernel<7, EB, CLUSTER>;
        case 8: return rs_square_kernel<8, EB, CLUSTER>;
        default: return rs_square_kernel<0, EB, CLUSTER>;
    }
}

// CTAs an SM up to which clip_adamw_kernel works its factor out itself, a launch less
// and some hundred clocks more a CTA: the clipped step of 700 K elements (2.3 CTAs an SM)
// takes 13.9 us so and 16.4 with norm_kernel; at 1.7 M both take 17.0, at 60 M
// norm_kernel saves 1 %.
constexpr int kSelfCtas = 4;

template <bool SELF>
auto pick_adamw(int eb, bool master) {
    return eb == 2 ? (master ? clip_adamw_kernel<2, true, SELF> : clip_adamw_kernel<2, false, SELF>)
                   : (master ? clip_adamw_kernel<4, true, SELF> : clip_adamw_kernel<4, false, SELF>);
}

}  // namespace

extern "C" {

int ss_grad_norm(int num_tensors, const int64_t* numels, const int* elem_bytes, const void* const* grads,
                 float* norm_out, void* workspace, size_t workspace_bytes, ss_stream_t stream) {
    if (!norm_out) return SS_EINVAL;
    if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
    if (!ss::aligned(norm_out, 4)) return SS_EALIGN;
    if (int rc = check_list(num_tensors, numels, elem_bytes, grads, nullptr)) return rc;
    return list_call(num_tensors, numels, elem_bytes, grads, nullptr, false, kNormOnly, norm_out, workspace,
                     reinterpret_cast<cudaStream_t>(stream));
}

int ss_clip_grads(int num_tensors, const int64_t* numels, const int* elem_bytes, void* const* grads,
                  void* const* out, double max_norm, float* norm_out, void* workspace,
                  size_t workspace_bytes, ss_stream_t stream) {
    if (!norm_out || !(max_norm >= 0.0)) return SS_EINVAL;
    if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
    if (!ss::aligned(norm_out, 4)) return SS_EALIGN;
    if (int rc = check_list(num_tensors, numels, elem_bytes, grads, out)) return rc;
    return list_call(num_tensors, numels, elem_bytes, grads, out, true, max_norm, norm_out, workspace,
                     reinterpret_cast<cudaStream_t>(stream));
}

int fsdp_reduce_scatter_norm(const ss_plan* plan, const void* const* rank_grads, float* reduced_grad,
                             double* sq_out, void* workspace, size_t workspace_bytes, int group,
                             ss_stream_t stream) {
    if (!plan || !rank_grads || !reduced_grad || !sq_out) return SS_EINVAL;
    if (!plan->has_dev) return SS_ENODEVICE;
    if (int rc = ss::check_device(plan)) return rc;
    if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
    int64_t lo, hi;
    if (!ss::group_range(plan, group, &lo, &hi)) return SS_EINVAL;
    RankPtrs rp;
    std::memset(&rp, 0, sizeof rp);
    for (int r = 0; r < plan->N; ++r) {
        if (!rank_grads[r] && hi > lo) return SS_EINVAL;
        if (!ss::aligned(rank_grads[r], 16)) return SS_EALIGN;
        rp.p[r] = rank_grads[r];
    }
    if (!ss::aligned(reduced_grad, 16) || !ss::aligned(sq_out, 8)) return SS_EALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const Split s = split_range(lo, hi > lo ? hi : lo, 16 / plan->eb);
    const int64_t per = s.nvec > 0 ? (s.nvec + kThreads - 1) / kThreads : 1;  // CTA rounds
    if (per <= 2 * kClusterMax) {
        auto fn = plan->eb == 2 ? pick_square<2, true>(plan->N) : pick_square<4, true>(plan->N);
        const int cluster = cluster_for(per);
        return ss::launch(fn, cluster, kThreads, 0, cluster, true, st, rp, plan->N, s,
                          (int)((per + cluster - 1) / cluster), reduced_grad, nullptr, sq_out);
    }
    const int64_t rounds = (per + kMaxPartials - 1) / kMaxPartials;
    if (rounds > INT32_MAX) return SS_EOVERFLOW;
    const int64_t n = (per + rounds - 1) / rounds;
    auto fn = plan->eb == 2 ? pick_square<2, false>(plan->N) : pick_square<4, false>(plan->N);
    if (int rc = ss::launch(fn, n, kThreads, 0, 0, true, st, rp, plan->N, s, (int)rounds, reduced_grad,
                            static_cast<float*>(workspace), nullptr))
        return rc;
    return fold(workspace, n, kNormOnly, sq_out, nullptr, st);
}

int fsdp_clip_adamw(const ss_plan* plan, const float* reduced_grad, const double* sq_sums, int num_sums,
                    double max_norm, float* master, float* exp_avg, float* exp_avg_sq, void* param_shards,
                    const ss_adamw* hp, float* norm_out, int group, ss_stream_t stream) {
    if (!plan || !reduced_grad || !sq_sums || num_sums < 1 || !(max_norm >= 0.0) || !exp_avg ||
        !exp_avg_sq || !param_shards || !hp || !norm_out)
        return SS_EINVAL;
    if (!plan->has_dev) return SS_ENODEVICE;
    if (int rc = ss::check_device(plan)) return rc;
    if (!ss::valid_hyper(hp)) return SS_EINVAL;
    int64_t lo, hi;
    if (!ss::group_range(plan, group, &lo, &hi)) return SS_EINVAL;
    const void* bufs[5] = {reduced_grad, master, exp_avg, exp_avg_sq, param_shards};
    for (const void* b : bufs)
        if (b && !ss::aligned(b, 16)) return SS_EALIGN;
    if (!ss::aligned(sq_sums, 8) || !ss::aligned(norm_out, 4)) return SS_EALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const AdamCoef c = ss::make_coef(hp);
    const Split s = split_range(lo, hi > lo ? hi : lo, 16 / plan->eb);
    const int64_t grid = s.nvec > 0 ? (s.nvec + kThreads - 1) / kThreads : 1;
    unsigned char* shards = static_cast<unsigned char*>(param_shards);
    if (grid <= (int64_t)ss::num_sms() * kSelfCtas)
        return ss::launch(pick_adamw<true>(plan->eb, master), grid, kThreads, 0, 0, true, st, reduced_grad, sq_sums,
                          num_sums, max_norm, norm_out, s, master, exp_avg, exp_avg_sq, shards, c);
    if (int rc = ss::launch(norm_kernel, 1, 32, 0, 0, true, st, sq_sums, num_sums, max_norm, norm_out)) return rc;
    return ss::launch(pick_adamw<false>(plan->eb, master), grid, kThreads, 0, 0, true, st, reduced_grad, sq_sums,
                      num_sums, max_norm, norm_out, s, master, exp_avg, exp_avg_sq, shards, c);
}

}  // extern "C"
