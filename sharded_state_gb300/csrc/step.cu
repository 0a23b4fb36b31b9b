// step.cu -- the whole sharded step in one pass over the parameters:
// (copy-in) + reduce-scatter + AdamW + (all-gather + unpack).
//
// fsdp_reduce_scatter_adamw streams the packed index space and
// fsdp_all_gather_unpack then reads the new shards back to unpack them.  The
// kernels here know for every element both its packed index f (gradient
// buffers, optimizer state, shards) and its place k inside the parameter
// tensor ("FSDP1 vs FSDP2" section 03 / 04: a run of one parameter inside one
// rank's shard).  The kernels stream f like the reduce-scatter and place
// each vector through the plan's packed segment map:
// fused_step_flat_kernel and, for the copy-in, its rounds form
// fused_step_flat_rounds_kernel when the runs are all whole 16-byte vectors;
// fused_step_flat_any_kernel (packed gradients) and
// fused_step_copyin_staged_kernel (per-parameter gradients, staged through
// shared memory) at any alignment.
// Per-parameter pointers ride in the kernel parameters; when a call's
// parameters need more than one table, each window of parameters runs over
// the packed ranges its segments form.  That lets one pass
//   - read the N gradients either from the packed rank buffers (the
//     reduce-scatter input FSDP builds by copy-in) or directly from the N
//     per-parameter gradient sets, which fuses the copy-in away;
//   - sum them in fp32 in rank order and divide by N (the reduce-scatter,
//     "Scaling data parallel" sections 9.1-9.3);
//   - run AdamW on the fp32 master and moments and write the bf16 shard;
//   - write the same bf16 value into the n_out per-parameter outputs (the
//     all-gather + unpack, "FSDP1 vs FSDP2" section 04), with no second pass
//     over the shards.
// Bytes per parameter element at N ranks: 2N (grads) + 12 + 12 (state) + 2
// (shard) + 2*n_out, e.g. 44 at N = 8, n_out = 1, against 46 for the two
// separate calls and 46 + 4N with a separate pack pass.  Pad elements are not
// touched: they hold zero gradients and zero state, which AdamW leaves zero.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <utility>
#include <vector>

#include "adamw.cuh"
#include "device_utils.cuh"
#include "internal.h"
#include "segmap.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTab = 2048;
constexpr int kMaxVec = 8;  // gradient vectors kept in flight per thread (ranks 0..7)
constexpr int kCopyinIters = 8;   // most rounds of vectors per warp in the copy-in kernels
constexpr int kCopyinWaves = 16;  // fewest waves of CTAs (3 per SM) the aligned copy-in keeps
constexpr int kCopyinMinWaves = 2;  // fewest waves of CTAs the staged copy-in keeps
constexpr int kFlatRounds = 4;    // most rounds per warp of the aligned flat copy-in

struct RankPtrs {
    const void* p[SS_MAX_WORLD];
};
template <int S>
struct PtrTabT {
    void* p[S];
};
using PtrTab = PtrTabT<kTab>;
// The table of small launches (see fsdp_sharded_step): 2 KiB of kernel
// parameters instead of 16 KiB, which a launch pays for on the host.
constexpr int kTabSmall = 256;
using PtrTabSmall = PtrTabT<kTabSmall>;
// Launches of at most this many vectors with a table that fits kTabSmall slots
// take the small form of the flat kernel.
constexpr int64_t kSmallVecs = (int64_t)2 * 3 * 152 * 256;
using ss::AdamCoef;
using ss::adamw_elem;
using ss::make_coef;

// Kernel arguments that do not change within a launch.
struct StepArgs {
    RankPtrs packed_grads;  // [N] packed rank buffers (UNPACKED == false)
    float* master;
    float* exp_avg;
    float* exp_avg_sq;
    uint16_t* shards;
    float* gout;
    int N;
    int n_out;
    int param_base;  // first parameter of this launch's window
    int w;           // parameters in the window
    int congruent;   // per-parameter gradients: every rank's pointer of every
                     // parameter in the window has the same address mod 16
    int M;           // entries of the packed segment map
    AdamCoef c;
};

// Table layout: UNPACKED gradients tab[r*w + slot] for r < N, then outputs
// tab[goff + j*w + slot] with goff = (UNPACKED ? N*w : 0).
template <bool UNPACKED, class Tab>
__device__ __forceinline__ const uint16_t* grad_ptr(const StepArgs& a, const Tab& tab, int r,
                                                    int slot, int64_t f, int64_t k) {
    if (UNPACKED) return static_cast<const uint16_t*>(tab.p[r * a.w + slot]) + k;
    return static_cast<const uint16_t*>(a.packed_grads.p[r]) + f;
}

// Rank-order fp32 sum of the first min(n, 8) ranks' vectors, from rank 0's value.
template <int NR>
__device__ __forceinline__ void sum_ranks(const uint4 (&w)[kMaxVec], int n, float (&s)[8]) {
    s[0] = ss::bf16_lo(w[0].x); s[1] = ss::bf16_hi(w[0].x);
    s[2] = ss::bf16_lo(w[0].y); s[3] = ss::bf16_hi(w[0].y);
    s[4] = ss::bf16_lo(w[0].z); s[5] = ss::bf16_hi(w[0].z);
    s[6] = ss::bf16_lo(w[0].w); s[7] = ss::bf16_hi(w[0].w);
#pragma unroll
    for (int r = 1; r < kMaxVec; ++r) {
        if (r < n) {
            s[0] = __fadd_rn(s[0], ss::bf16_lo(w[r].x));
            s[1] = __fadd_rn(s[1], ss::bf16_hi(w[r].x));
            s[2] = __fadd_rn(s[2], ss::bf16_lo(w[r].y));
            s[3] = __fadd_rn(s[3], ss::bf16_hi(w[r].y));
            s[4] = __fadd_rn(s[4], ss::bf16_lo(w[r].z));
            s[5] = __fadd_rn(s[5], ss::bf16_hi(w[r].z));
            s[6] = __fadd_rn(s[6], ss::bf16_lo(w[r].w));
            s[7] = __fadd_rn(s[7], ss::bf16_hi(w[r].w));
        }
    }
}

__device__ __forceinline__ void add_rank(float (&s)[8], uint4 x) {
    s[0] = __fadd_rn(s[0], ss::bf16_lo(x.x));
    s[1] = __fadd_rn(s[1], ss::bf16_hi(x.x));
    s[2] = __fadd_rn(s[2], ss::bf16_lo(x.y));
    s[3] = __fadd_rn(s[3], ss::bf16_hi(x.y));
    s[4] = __fadd_rn(s[4], ss::bf16_lo(x.z));
    s[5] = __fadd_rn(s[5], ss::bf16_hi(x.z));
    s[6] = __fadd_rn(s[6], ss::bf16_lo(x.w));
    s[7] = __fadd_rn(s[7], ss::bf16_hi(x.w));
}

// Ranks 8 .. n-1 (N > 8) added to s in rank order, 8 loads in flight at a
// time in w (free once the first 8 ranks are summed).
template <bool UNPACKED, class Tab>
__device__ __forceinline__ void add_ranks_beyond_8(const StepArgs& a, const Tab& tab, int slot,
                                                   int64_t f, int64_t k, int n,
                                                   uint4 (&w)[kMaxVec], float (&s)[8]) {
    for (int r0 = kMaxVec; r0 < n; r0 += kMaxVec) {
#pragma unroll
        for (int j = 0; j < kMaxVec; ++j)
            if (r0 + j < n) w[j] = ss::ld_stream_u4(grad_ptr<UNPACKED>(a, tab, r0 + j, slot, f, k));
#pragma unroll
        for (int j = 0; j < kMaxVec; ++j)
            if (r0 + j < n) add_rank(s, w[j]);
    }
}

// The rank sum s of 8 elements divided by n (g) and AdamW on the state loaded
// as t/m/v, giving the new master, moments th/mm/vv.
__device__ __forceinline__ void adam_compute(const StepArgs& a, const float (&s)[8], int n, float4 t0,
                                             float4 t1, float4 m0, float4 m1, float4 v0, float4 v1,
                                             float (&g)[8], float (&th)[8], float (&mm)[8],
                                             float (&vv)[8]) {
    const float fN = (float)n;
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = __fdiv_rn(s[e], fN);
    th[0] = t0.x; th[1] = t0.y; th[2] = t0.z; th[3] = t0.w;
    th[4] = t1.x; th[5] = t1.y; th[6] = t1.z; th[7] = t1.w;
    mm[0] = m0.x; mm[1] = m0.y; mm[2] = m0.z; mm[3] = m0.w;
    mm[4] = m1.x; mm[5] = m1.y; mm[6] = m1.z; mm[7] = m1.w;
    vv[0] = v0.x; vv[1] = v0.y; vv[2] = v0.z; vv[3] = v0.w;
    vv[4] = v1.x; vv[5] = v1.y; vv[6] = v1.z; vv[7] = v1.w;
#pragma unroll
    for (int e = 0; e < 8; ++e) adamw_elem(g[e], th[e], mm[e], vv[e], a.c);
}

// The rank sum s of packed elements f..f+7 divided by n, AdamW on the state
// loaded as t/m/v, state and shard stores (and the reduced gradient when
// a.gout is set); returns the new bf16 parameter vector.
__device__ __forceinline__ uint4 adam_vec(const StepArgs& a, int64_t f, const float (&s)[8], int n,
                                          float4 t0, float4 t1, float4 m0, float4 m1, float4 v0,
                                          float4 v1) {
    const float fN = (float)n;
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = __fdiv_rn(s[e], fN);
    if (a.gout) {
        ss::st_stream_f4(a.gout + f, make_float4(g[0], g[1], g[2], g[3]));
        ss::st_stream_f4(a.gout + f + 4, make_float4(g[4], g[5], g[6], g[7]));
    }
    float th[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
    float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
    float vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) adamw_elem(g[e], th[e], mm[e], vv[e], a.c);
    ss::st_stream_f4(a.master + f, make_float4(th[0], th[1], th[2], th[3]));
    ss::st_stream_f4(a.master + f + 4, make_float4(th[4], th[5], th[6], th[7]));
    ss::st_stream_f4(a.exp_avg + f, make_float4(mm[0], mm[1], mm[2], mm[3]));
    ss::st_stream_f4(a.exp_avg + f + 4, make_float4(mm[4], mm[5], mm[6], mm[7]));
    ss::st_stream_f4(a.exp_avg_sq + f, make_float4(vv[0], vv[1], vv[2], vv[3]));
    ss::st_stream_f4(a.exp_avg_sq + f + 4, make_float4(vv[4], vv[5], vv[6], vv[7]));
    uint4 p;
    p.x = ss::pack_bf16x2(th[0], th[1]);
    p.y = ss::pack_bf16x2(th[2], th[3]);
    p.z = ss::pack_bf16x2(th[4], th[5]);
    p.w = ss::pack_bf16x2(th[6], th[7]);
    ss::st_stream_u4(a.shards + f, p);
    return p;
}

template <bool UNPACKED, class Tab>
__device__ __forceinline__ void step_scalar(const StepArgs& a, const Tab& tab, int slot,
                                            int64_t f, int64_t k) {
    const int n = a.N;
    float s = ss::bf16_to_f32(*grad_ptr<UNPACKED>(a, tab, 0, slot, f, k));
    for (int r = 1; r < n; ++r) s = __fadd_rn(s, ss::bf16_to_f32(*grad_ptr<UNPACKED>(a, tab, r, slot, f, k)));
    const float g = __fdiv_rn(s, (float)n);
    if (a.gout) a.gout[f] = g;
    float th = a.master[f], m = a.exp_avg[f], v = a.exp_avg_sq[f];
    adamw_elem(g, th, m, v, a.c);
    a.master[f] = th;
    a.exp_avg[f] = m;
    a.exp_avg_sq[f] = v;
    const uint16_t p = ss::f32_to_bf16(th);
    a.shards[f] = p;
    const int goff = UNPACKED ? n * a.w : 0;
    for (int j = 0; j < a.n_out; ++j) static_cast<uint16_t*>(tab.p[goff + j * a.w + slot])[k] = p;
}

// Element x (index k of parameter slot) of a vector that meets a segment end,
// with per-parameter gradients: the rank-order sum of its N gradients (every
// rank's load issued before the adds, 8 at a time), then AdamW on
// the state values th/m/v loaded with the vector, and the stores.  The same
// operations as step_scalar.
template <int NR>
__device__ __forceinline__ void step_elem(const StepArgs& a, const PtrTab& tab, int slot, int64_t x,
                                          int64_t k, float th, float m, float v) {
    const int n = NR > 0 ? NR : a.N;
    constexpr int kB = kMaxVec;  // loads in flight
    float s = 0.f;
#pragma unroll
    for (int r0 = 0; r0 < (NR > 0 ? NR : n); r0 += kB) {
        uint16_t h[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j)
            if (r0 + j < n) h[j] = static_cast<const uint16_t*>(tab.p[(r0 + j) * a.w + slot])[k];
#pragma unroll
        for (int j = 0; j < kB; ++j)
            if (r0 + j < n) s = r0 + j == 0 ? ss::bf16_to_f32(h[j]) : __fadd_rn(s, ss::bf16_to_f32(h[j]));
    }
    const float g = __fdiv_rn(s, (float)n);
    if (a.gout) a.gout[x] = g;
    adamw_elem(g, th, m, v, a.c);
    a.master[x] = th;
    a.exp_avg[x] = m;
    a.exp_avg_sq[x] = v;
    const uint16_t p = ss::f32_to_bf16(th);
    a.shards[x] = p;
    const int goff = n * a.w;
    for (int j = 0; j < a.n_out; ++j) static_cast<uint16_t*>(tab.p[goff + j * a.w + slot])[k] = p;
}

// Flat form of the one-pass step, for plans whose runs are all whole 16-byte
// vectors with 16-byte aligned per-parameter pointers: thread q of the grid
// takes packed elements f = vbeg + 8q .. f + 7, as the reduce-scatter kernel
// does.  The state loads depend on f alone and go out first, and so do the
// gradient loads when the gradients are packed.  The segment holding f --
// needed for the per-parameter gradients (UNPACKED) and outputs -- is looked
// up meanwhile: the block index gives the segment that covers the start of
// f's kMapBlock block, which is f's own segment unless a segment starts
// inside the block; only then a binary search over the few segments that
// start in the block follows.  A pad vector is read (state, packed
// gradients) but nothing is stored.
// SMALL (launches of a few waves, whose time is mostly launch and latency):
// a 256-slot pointer table, and the kernel is launched with programmatic
// stream serialisation.  It lets the next launch on the stream start at once
// and looks its segment up -- the plan's map, which no kernel writes --
// before it waits (griddepcontrol.wait) for the grid before it on the stream
// to complete; only then does it touch state, gradients or outputs.  So
// back-to-back steps overlap one's launch and lookup with the previous one's
// end.  Without a programmatic predecessor the wait returns at once.
template <int NR, bool UNPACKED, bool SMALL = false>
__global__ void __launch_bounds__(kThreads, 3)
fused_step_flat_kernel(const ss::PmEntry* __restrict__ pm, const int* __restrict__ pm_block,
                       int64_t vbeg, int64_t nvec, StepArgs a,
                       PtrTabT<SMALL ? kTabSmall : kTab> tab) {
    if (SMALL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (q >= nvec) {
        if (SMALL) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int64_t f = vbeg + 8 * q;
    const int64_t B = f / ss::kMapBlock;
    int m = __ldg(pm_block + B);
    const int n = NR > 0 ? NR : a.N;
    ss::PmEntry e;
    if (SMALL) {  // the segment first, then the wait for the previous grid
        e = pm[m];
        ss::locate(ss::SegMap{pm, pm_block, 0}, B, f, m, e);
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    uint4 w[kMaxVec];
    if (!UNPACKED) {
#pragma unroll
        for (int r = 0; r < kMaxVec; ++r)
            if (r < n) w[r] = ss::ld_stream_u4(static_cast<const uint16_t*>(a.packed_grads.p[r]) + f);
    }
    // N > 8 (the general instance): the state is loaded after the ranks are
    // summed, so that its registers are not held across the rank batches
    constexpr bool kRanksFirst = NR == 0;
    float4 t0, t1, m0, m1, v0, v1;
    auto load_state = [&]() {
        t0 = ss::ld_rw_f4(a.master + f);
        t1 = ss::ld_rw_f4(a.master + f + 4);
        m0 = ss::ld_rw_f4(a.exp_avg + f);
        m1 = ss::ld_rw_f4(a.exp_avg + f + 4);
        v0 = ss::ld_rw_f4(a.exp_avg_sq + f);
        v1 = ss::ld_rw_f4(a.exp_avg_sq + f + 4);
    };
    if (!kRanksFirst) load_state();
    if (!SMALL) {
        e = pm[m];
        if (f < e.packed_off || f >= e.packed_off + e.len) {  // a segment starts inside the block
            int hi = __ldg(pm_block + B + 1);
            while (m < hi) {
                const int mid = (m + hi + 1) >> 1;
                if (pm[mid].packed_off <= f)
                    m = mid;
                else
                    hi = mid - 1;
            }
            e = pm[m];
        }
    }
    const int64_t rel = f - e.packed_off;
    if (rel < 0 || rel >= e.len) return;  // a pad vector
    const int slot = e.param - a.param_base;
    const int64_t k = e.param_off + rel;  // index inside the parameter tensor
    if (UNPACKED) {
#pragma unroll
        for (int r = 0; r < kMaxVec; ++r)
            if (r < n) w[r] = ss::ld_stream_u4(static_cast<const uint16_t*>(tab.p[r * a.w + slot]) + k);
    }
    float s[8];
    sum_ranks<NR>(w, n, s);
    if (NR == 0 || NR > kMaxVec) add_ranks_beyond_8<UNPACKED>(a, tab, slot, f, k, n, w, s);
    if (kRanksFirst) load_state();
    const uint4 p = adam_vec(a, f, s, n, t0, t1, m0, m1, v0, v1);
    const int goff = UNPACKED ? n * a.w : 0;
    for (int j = 0; j < a.n_out; ++j)
        ss::st_stream_u4(static_cast<uint16_t*>(tab.p[goff + j * a.w + slot]) + k, p);
}

// fused_step_flat_kernel with per-parameter gradients (the fused copy-in),
// in rounds: warp gw takes `iters` rounds of 32 consecutive packed vectors
// (lane = vector, as in the one-shot form).  The gradient loads wait for the
// vector's segment, so a lane keeps its segment from one round to the next
// (no lookup while it stays inside) and, once this round's loads are out,
// asks L2 for the next round's state and gradient lines: the next round's
// loads then wait for L2 rather than DRAM while this one computes.
template <int NR>  // 2..8
__global__ void __launch_bounds__(kThreads, 3)
fused_step_flat_rounds_kernel(const ss::PmEntry* __restrict__ pm, const int* __restrict__ pm_block,
                              int64_t vbeg, int64_t nvec, int iters, StepArgs a, PtrTab tab) {
    const ss::SegMap mp{pm, pm_block, 0};
    const int lane = threadIdx.x & 31;
    const int64_t gw = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    constexpr int n = NR;
    const int64_t fend = vbeg + 8 * nvec;
    int64_t hend = 0, hdelta = 0;  // the lane's last segment: its end and k - f
    int hslot = -1;                // and parameter slot (-1: none)
    int64_t f = vbeg + 8 * (gw * iters * 32 + lane);
    for (int it = iters; it > 0 && f < fend; --it, f += 8 * 32) {
        const float4 t0 = ss::ld_rw_f4(a.master + f), t1 = ss::ld_rw_f4(a.master + f + 4);
        const float4 m0 = ss::ld_rw_f4(a.exp_avg + f), m1 = ss::ld_rw_f4(a.exp_avg + f + 4);
        const float4 v0 = ss::ld_rw_f4(a.exp_avg_sq + f), v1 = ss::ld_rw_f4(a.exp_avg_sq + f + 4);
        if (hslot < 0 || f + 8 > hend) {  // leaves the last segment: look it up
            int m;
            const ss::PmEntry e = ss::lookup(mp, f, m);
            hslot = -1;
            if (f >= e.packed_off && f < e.packed_off + e.len) {
                hend = e.packed_off + e.len;
                hdelta = e.param_off - e.packed_off;
                hslot = e.param - a.param_base;
            }
        }
        const int64_t fn = f + 8 * 32;
        const bool next = it > 1 && fn < fend;
        if (next) {
            ss::prefetch_l2(a.master + fn);
            ss::prefetch_l2(a.exp_avg + fn);
            ss::prefetch_l2(a.exp_avg_sq + fn);
        }
        if (hslot < 0) continue;  // a pad vector
        const int slot = hslot;
        const int64_t k = f + hdelta;  // index inside the parameter tensor
        uint4 w[kMaxVec];
#pragma unroll
        for (int r = 0; r < kMaxVec; ++r)
            if (r < n) w[r] = ss::ld_stream_u4(static_cast<const uint16_t*>(tab.p[r * a.w + slot]) + k);
        if (next && fn + 8 <= hend) {
#pragma unroll
            for (int r = 0; r < kMaxVec; ++r)
                if (r < n) ss::prefetch_l2(static_cast<const uint16_t*>(tab.p[r * a.w + slot]) + fn + hdelta);
        }
        float s[8];
        sum_ranks<NR>(w, n, s);
        const uint4 p = adam_vec(a, f, s, n, t0, t1, m0, m1, v0, v1);
        const int goff = n * a.w;
        for (int j = 0; j < a.n_out; ++j)
            ss::st_stream_u4(static_cast<uint16_t*>(tab.p[goff + j * a.w + slot]) + k, p);
    }
}

using FlatRoundsKern = void (*)(const ss::PmEntry*, const int*, int64_t, int64_t, int, StepArgs,
                                PtrTab);

FlatRoundsKern pick_flat_rounds(int N) {
    switch (N) {
        case 2: return fused_step_flat_rounds_kernel<2>;
        case 3: return fused_step_flat_rounds_kernel<3>;
        case 4: return fused_step_flat_rounds_kernel<4>;
        case 5: return fused_step_flat_rounds_kernel<5>;
        case 6: return fused_step_flat_rounds_kernel<6>;
        case 7: return fused_step_flat_rounds_kernel<7>;
        case 8: return fused_step_flat_rounds_kernel<8>;
        default: return nullptr;  // the one-shot form
    }
}

using FlatKern = void (*)(const ss::PmEntry*, const int*, int64_t, int64_t, StepArgs, PtrTab);
using FlatKernSmall = void (*)(const ss::PmEntry*, const int*, int64_t, int64_t, StepArgs,
                               PtrTabSmall);

template <bool U, bool SMALL = false>
auto pick_flat(int N) {
    switch (N) {
        case 1: return fused_step_flat_kernel<1, U, SMALL>;
        case 2: return fused_step_flat_kernel<2, U, SMALL>;
        case 3: return fused_step_flat_kernel<3, U, SMALL>;
        case 4: return fused_step_flat_kernel<4, U, SMALL>;
        case 5: return fused_step_flat_kernel<5, U, SMALL>;
        case 6: return fused_step_flat_kernel<6, U, SMALL>;
        case 7: return fused_step_flat_kernel<7, U, SMALL>;
        case 8: return fused_step_flat_kernel<8, U, SMALL>;
        default: return fused_step_flat_kernel<0, U, SMALL>;
    }
}

// The n_out per-parameter outputs of one vector p at index k of parameter
// `slot` (output j at tab[goff + j*w + slot]), sh bytes past a 16-byte
// boundary: the aligned block after the vector's start is written whole
// (this vector's last sh bytes, then the first 16 - sh of nx, the next
// vector of the same run) when same_next, else only this vector's bytes of
// it; unless same_prev (the previous vector of the run writes the block
// before whole), the vector's first 16 - sh bytes go into the block before.
template <class Tab>
__device__ __forceinline__ void store_outputs_lane(const StepArgs& a, const Tab& tab, int goff,
                                                   int slot, int64_t k, uint4 p, uint4 nx,
                                                   bool same_next, bool same_prev) {
    for (int j = 0; j < a.n_out; ++j)
        ss::store_realigned(
            reinterpret_cast<unsigned char*>(static_cast<uint16_t*>(tab.p[goff + j * a.w + slot]) + k), p,
            nx, same_next, same_prev);
}

// The call range's elements outside whole packed vectors: [h0, h0 + nh) at
// its start and [t0, t0 + nt) at its end, fewer than 8 each.
struct EdgeElems {
    int64_t h0, t0;
    int nh, nt;
};

// Flat form of the one-pass step for packed gradients at any alignment of the
// runs and of the per-parameter outputs.  Thread q takes the 8-aligned packed
// vector f = vbeg + 8q; its gradient and state loads are aligned and go out
// before the segment lookup, as in the aligned flat kernel.
//  - A vector inside one segment (the common case) stores its state and shard
//    as vectors.  Its per-parameter output starts sh bytes past a 16-byte
//    boundary; when the next lane holds the next vector of the same segment,
//    the lane writes the aligned block after its start whole (its last sh
//    bytes, the next vector's first 16 - sh), otherwise only its own bytes of
//    that block; a lane whose previous lane is not its predecessor in the
//    segment also writes its first 16 - sh bytes into the block before.
//  - A vector that meets a segment end (the rest pad or the next segment's
//    start) is stored element by element, each element placed by its own
//    segment; pad elements are not stored.
//  - Threads nvec .. nvec + 15 take the range's edge elements one by one.
// Lanes never leave before the shuffles, so whole warps take part in them.
template <int NR, bool SMALL = false>
__global__ void __launch_bounds__(kThreads, 3)
fused_step_flat_any_kernel(const ss::PmEntry* __restrict__ pm, const int* __restrict__ pm_block,
                           int M, int64_t vbeg, int64_t nvec, EdgeElems ed, StepArgs a,
                           PtrTabT<SMALL ? kTabSmall : kTab> tab) {
    if (SMALL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const ss::SegMap mp{pm, pm_block, M};
    const int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int lane = threadIdx.x & 31;
    const int n = NR > 0 ? NR : a.N;
    int key = -1;  // map entry of a vector inside one segment, else -1
    int slot = 0;
    int64_t k = 0;
    uint4 p = make_uint4(0, 0, 0, 0);
    if (q < nvec) {
        const int64_t f = vbeg + 8 * q;
        const int64_t B = f / ss::kMapBlock;
        int m = __ldg(mp.pm_block + B);
        ss::PmEntry e;
        if (SMALL) {  // the segment first, then the wait for the previous grid
            e = mp.pm[m];
            ss::locate(mp, B, f, m, e);
            asm volatile("griddepcontrol.wait;" ::: "memory");
        }
        uint4 w[kMaxVec];
#pragma unroll
        for (int r = 0; r < kMaxVec; ++r)
            if (r < n) w[r] = ss::ld_stream_u4(static_cast<const uint16_t*>(a.packed_grads.p[r]) + f);
        float s[8];
        // N > 8: the ranks are summed before the state is loaded, so that the
        // state's registers are not held across the rank batches (without
        // it the general instance spills)
        constexpr bool kRanksFirst = NR == 0 || NR > kMaxVec;
        if (kRanksFirst) {
            sum_ranks<NR>(w, n, s);
            add_ranks_beyond_8<false>(a, tab, 0, f, 0, n, w, s);
        }
        const float4 t0 = ss::ld_rw_f4(a.master + f), t1 = ss::ld_rw_f4(a.master + f + 4);
        const float4 m0 = ss::ld_rw_f4(a.exp_avg + f), m1 = ss::ld_rw_f4(a.exp_avg + f + 4);
        const float4 v0 = ss::ld_rw_f4(a.exp_avg_sq + f), v1 = ss::ld_rw_f4(a.exp_avg_sq + f + 4);
        if (!SMALL) {
            e = mp.pm[m];
            ss::locate(mp, B, f, m, e);
        }
        if (!kRanksFirst) {
            sum_ranks<NR>(w, n, s);
            if (NR == 0 || NR > kMaxVec) add_ranks_beyond_8<false>(a, tab, 0, f, 0, n, w, s);
        }
        if (f >= e.packed_off && f + 8 <= e.packed_off + e.len) {
            p = adam_vec(a, f, s, n, t0, t1, m0, m1, v0, v1);
            key = m;
            slot = e.param - a.param_base;
            k = e.param_off + (f - e.packed_off);
        } else {
            float g[8], th[8], mm[8], vv[8];
            adam_compute(a, s, n, t0, t1, m0, m1, v0, v1, g, th, mm, vv);
            const int goff = 0;
            int c = m;  // the entry of element f + i: the last one starting at or before it
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t x = f + i;
                while (c + 1 < mp.M && mp.pm[c + 1].packed_off <= x) {
                    ++c;
                    e = mp.pm[c];
                }
                if (x < e.packed_off || x >= e.packed_off + e.len) continue;  // pad
                if (a.gout) a.gout[x] = g[i];
                a.master[x] = th[i];
                a.exp_avg[x] = mm[i];
                a.exp_avg_sq[x] = vv[i];
                const uint16_t b = ss::f32_to_bf16(th[i]);
                a.shards[x] = b;
                const int sl = e.param - a.param_base;
                const int64_t kx = e.param_off + (x - e.packed_off);
                for (int j = 0; j < a.n_out; ++j)
                    static_cast<uint16_t*>(tab.p[goff + j * a.w + sl])[kx] = b;
            }
        }
    }
    const int nkey = __shfl_down_sync(0xFFFFFFFFu, key, 1);
    const int pkey = __shfl_up_sync(0xFFFFFFFFu, key, 1);
    uint4 nx;
    nx.x = __shfl_down_sync(0xFFFFFFFFu, p.x, 1);
    nx.y = __shfl_down_sync(0xFFFFFFFFu, p.y, 1);
    nx.z = __shfl_down_sync(0xFFFFFFFFu, p.z, 1);
    nx.w = __shfl_down_sync(0xFFFFFFFFu, p.w, 1);
    if (key >= 0) store_outputs_lane(a, tab, 0, slot, k, p, nx, lane < 31 && nkey == key,
                                     lane > 0 && pkey == key);
    if (q >= nvec && q < nvec + 16) {
        const int i = (int)(q - nvec);
        if (i < 8 ? i < ed.nh : i - 8 < ed.nt) {
            const int64_t x = i < 8 ? ed.h0 + i : ed.t0 + (i - 8);
            int m;
            const ss::PmEntry e = ss::lookup(mp, x, m);
            if (SMALL) asm volatile("griddepcontrol.wait;" ::: "memory");
            if (x >= e.packed_off && x < e.packed_off + e.len)
                step_scalar<false>(a, tab, e.param - a.param_base, x, e.param_off + (x - e.packed_off));
        }
    }
}

// Shared-memory staging of the fused copy-in: per warp, rank and round, the
// aligned 16-byte blocks that cover the warp's 32 vectors (33 when the
// gradient tensor's run is not 16-byte aligned), ranks in batches of 8.
constexpr int kStageBlocks = 33;
constexpr int kStageBatch = 8;
constexpr int kStagedWarps = kThreads / 32;

__host__ __device__ constexpr int staged_bufs(int NR) { return NR > 0 && NR <= kStageBatch ? 1 : 2; }
__host__ __device__ constexpr int staged_smem_bytes(int NR) {
    return kStagedWarps * staged_bufs(NR) * kStageBatch * kStageBlocks * 16;
}

// Element E (0..15) of the 32 bytes x0:x1 as fp32: the low or high half of
// word E / 2 (bf16 -> fp32 is exact).
template <int E>
__device__ __forceinline__ float elem_at(const uint4& x0, const uint4& x1) {
    constexpr int w = E >> 1;
    const uint32_t v = w == 0 ? x0.x : w == 1 ? x0.y : w == 2 ? x0.z : w == 3 ? x0.w
                     : w == 4 ? x1.x : w == 5 ? x1.y : w == 6 ? x1.z : x1.w;
    return (E & 1) ? ss::bf16_hi(v) : ss::bf16_lo(v);
}

// A lane's 8 gradient elements of one rank, read from its staged blocks
// blk[0], blk[1] at element offset H (the run's address mod 16, over 2),
// added to s in rank order (FIRST: rank 0, s starts from its values).
template <int H, bool FIRST>
__device__ __forceinline__ void add_staged(float (&s)[8], const uint4* blk) {
    const uint4 x0 = blk[0];
    const uint4 x1 = H ? blk[1] : x0;
#define SS_ADD_STAGED(E)                                   \
    {                                                      \
        const float v = elem_at<H + E>(x0, x1);            \
        s[E] = FIRST ? v : __fadd_rn(s[E], v);             \
    }
    SS_ADD_STAGED(0) SS_ADD_STAGED(1) SS_ADD_STAGED(2) SS_ADD_STAGED(3)
    SS_ADD_STAGED(4) SS_ADD_STAGED(5) SS_ADD_STAGED(6) SS_ADD_STAGED(7)
#undef SS_ADD_STAGED
}

// The rank sum of one round of the staged copy-in, every vector of the warp
// inside one segment: rank r's gradient bytes of the warp are the run at
// tab[r][slot0] + k0 of 8 * nl elements.  The aligned 16-byte blocks that
// cover it go to shared memory by cp.async (lane l block l, lane 0 also the
// 33rd), ranks in batches of 8 (two in flight above N = 8; a buffer is
// refilled only after every lane has read it); each lane then reads its own
// two blocks back and adds its 8 elements to s in rank order, from rank 0's
// value.  H >= 0: every rank's run sits at element offset H of its first
// block (the host checked the pointers' addresses mod 16), so the elements
// are picked straight out of the two blocks; H = -1: each rank's own offset,
// realigned with funnel shifts.  prefetch_next runs once the first copies
// are out.
template <int NR, int H, typename Pre>
__device__ __forceinline__ void staged_sum(const StepArgs& a, const PtrTab& tab, int slot0,
                                           int64_t k0, int nl, int lane, uint32_t wst_s,
                                           const uint4* wst, float (&s)[8], Pre prefetch_next) {
    constexpr int kBufBlocks = kStageBatch * kStageBlocks;
    const int n = NR > 0 ? NR : a.N;
    const int nbat = (n + kStageBatch - 1) / kStageBatch;
    auto run = [&](int r) {
        return reinterpret_cast<const unsigned char*>(static_cast<const uint16_t*>(tab.p[r * a.w + slot0]) +
                                                      k0);
    };
    auto issue = [&](int b) {
        const uint32_t buf = wst_s + (uint32_t)((b % staged_bufs(NR)) * kBufBlocks * 16);
#pragma unroll
        for (int j = 0; j < kStageBatch; ++j) {
            const int r = b * kStageBatch + j;
            if (r < n) {
                const unsigned char* g = run(r);
                const int sh = H >= 0 ? 2 * H : (int)(reinterpret_cast<uintptr_t>(g) & 15u);
                const unsigned char* base = g - sh;
                const int nblk = nl + (sh ? 1 : 0);
                const uint32_t dst = buf + (uint32_t)(j * kStageBlocks * 16);
                if (lane < nblk) ss::cp_async16(dst + 16 * lane, base + 16 * lane);
                if (lane + 32 < nblk) ss::cp_async16(dst + 16 * (lane + 32), base + 16 * (lane + 32));
            }
        }
        ss::cp_async_commit();
    };
    __syncwarp();  // every lane has read the last round's buffers
    issue(0);
    if (nbat > 1) issue(1);
    prefetch_next();
    for (int b = 0; b < nbat; ++b) {
        if (b + 1 < nbat)
            ss::cp_async_wait<1>();
        else
            ss::cp_async_wait<0>();
        __syncwarp();
        const uint4* buf = wst + (b % staged_bufs(NR)) * kBufBlocks;
#pragma unroll
        for (int j = 0; j < kStageBatch; ++j) {
            const int r = b * kStageBatch + j;
            if (r < n && lane < nl) {
                const uint4* blk = buf + j * kStageBlocks + lane;
                if constexpr (H >= 0) {
                    if (r == 0)
                        add_staged<H, true>(s, blk);
                    else
                        add_staged<H, false>(s, blk);
                } else {
                    const int sh = (int)(reinterpret_cast<uintptr_t>(run(r)) & 15u);
                    uint4 x = blk[0];
                    if (sh) x = ss::realign16(x, blk[1], sh);
                    if (r == 0) {
                        s[0] = ss::bf16_lo(x.x); s[1] = ss::bf16_hi(x.x);
                        s[2] = ss::bf16_lo(x.y); s[3] = ss::bf16_hi(x.y);
                        s[4] = ss::bf16_lo(x.z); s[5] = ss::bf16_hi(x.z);
                        s[6] = ss::bf16_lo(x.w); s[7] = ss::bf16_hi(x.w);
                    } else {
                        add_rank(s, x);
                    }
                }
            }
        }
        if (b + 2 < nbat) {
            __syncwarp();  // every lane has read the buffer it refills
            issue(b + 2);
        }
    }
}

// Flat form of the one-pass step with per-parameter gradients (fused
// copy-in) at any alignment of the runs and the pointers, for any N, in one
// pass.  A CTA takes 8 * iters rounds of 32 consecutive 8-aligned packed
// vectors, lane = vector, and its warp wib every 8th of them from round wib,
// so that the CTA's warps read neighbouring runs at once; a lane keeps the
// segment of its last vector and looks it up in the packed segment map only
// when it leaves it.  When every
// vector of the round lies in one segment (all but the rounds that meet a
// segment end), the warp's gradient bytes of rank r are one contiguous run of
// the rank's tensor: the warp copies the aligned 16-byte blocks covering it
// into shared memory with cp.async -- lane l block l, lane 0 also the 33rd --
// so nothing is held in registers per rank, and each lane reads its own 16
// bytes back from its two blocks, shifted into place.  Ranks go in batches of
// 8 (NR = N <= 8: one batch); with more, two batches are in flight while the
// earlier one is summed, and a buffer is refilled only after every lane has
// read it.  The sum runs in rank order from rank 0's value, as everywhere.
// Rounds that meet a segment end load each vector inside one segment
// straight from global memory (ld_any16) and run the others element by
// element.  Every block read holds at least one byte of the run, so no load
// leaves the gradient tensor's 16-byte blocks.  Outputs as in
// fused_step_flat_any_kernel.  One launch takes all the runs of one pointer
// table (StagedRuns: with the per-parameter layout a window of parameters
// cut out of a group is one run per rank shard); each run has its own CTAs,
// and its edge elements run on lanes 0..15 of the warp after its rounds'.
// The runs of one staged copy-in launch: a parameter window's runs of the
// packed index (at most kMaxRuns), run i its whole vectors [vbeg[i], vbeg[i] +
// 8 * nvec[i]), taken by nwarps[i] warps of `iters` rounds, and its edge
// elements ed[i] (on the warp after them); run i takes CTAs [cta0[i],
// cta0[i + 1]).
constexpr int kMaxRuns = 64;
struct StagedRuns {
    int64_t vbeg[kMaxRuns];
    int64_t nvec[kMaxRuns];
    int64_t nwarps[kMaxRuns];
    int64_t cta0[kMaxRuns + 1];
    EdgeElems ed[kMaxRuns];
    int n;
};

template <int NR>
__global__ void __launch_bounds__(kThreads, 3)
fused_step_copyin_staged_kernel(const ss::PmEntry* __restrict__ pm, const int* __restrict__ pm_block,
                                StagedRuns runs, int iters, int pdl, StepArgs a, PtrTab tab) {
    extern __shared__ uint4 stage[];
    // pdl bit 0: the call's next staged launch (another window's runs) may
    // start once every CTA here has; bit 1: this launch ends only after the
    // one before it (programmatic dependent launch: the launches touch
    // disjoint elements, and a following kernel still sees both done)
    if (pdl & 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const ss::SegMap mp{pm, pm_block, 0};
    constexpr unsigned kAll = 0xFFFFFFFFu;
    constexpr int kBufBlocks = kStageBatch * kStageBlocks;  // one batch of ranks
    const int lane = threadIdx.x & 31;
    const int wib = threadIdx.x >> 5;
    int ri = 0;  // the CTA's run
    while (ri + 1 < runs.n && (int64_t)blockIdx.x >= runs.cta0[ri + 1]) ++ri;
    const int64_t cb = (int64_t)blockIdx.x - runs.cta0[ri];  // the CTA's place in its run
    const int64_t vbeg = runs.vbeg[ri], nvec = runs.nvec[ri], nwarps = runs.nwarps[ri];
    const EdgeElems ed = runs.ed[ri];
    const int64_t gw = cb * kStagedWarps + wib;
    const int n = NR > 0 ? NR : a.N;
    const uint4* wst = stage + (size_t)wib * staged_bufs(NR) * kBufBlocks;
    const uint32_t wst_s = (uint32_t)__cvta_generic_to_shared(wst);
    const int goff = n * a.w;
    const int64_t fend = vbeg + 8 * nvec;
    int64_t hend = 0, hdelta = 0;  // the lane's last segment: its end and k - f,
    int hslot = 0, hkey = -1;      // its parameter slot and map index (-1: none)
    // the CTA's 8 * iters rounds, interleaved: warp wib takes rounds wib,
    // wib + 8, ... of them, so the CTA's warps read neighbouring 512-byte runs
    // of each rank at once (4 KiB together) rather than runs 8 rounds apart
    constexpr int64_t kStride = 8 * 32 * kStagedWarps;  // elements between a warp's rounds
    int64_t f = vbeg + 8 * ((cb * kStagedWarps * iters + wib) * 32 + lane);
    for (int it = iters; it > 0; --it, f += kStride) {
        if (__shfl_sync(kAll, f, 0) >= fend) break;  // the same for the whole warp
        const bool has = f < fend;
        const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 t0 = z4, t1 = z4, m0 = z4, m1 = z4, v0 = z4, v1 = z4;
        if (has) {
            t0 = ss::ld_rw_f4(a.master + f);
            t1 = ss::ld_rw_f4(a.master + f + 4);
            m0 = ss::ld_rw_f4(a.exp_avg + f);
            m1 = ss::ld_rw_f4(a.exp_avg + f + 4);
            v0 = ss::ld_rw_f4(a.exp_avg_sq + f);
            v1 = ss::ld_rw_f4(a.exp_avg_sq + f + 4);
        }
        if (has && (hkey < 0 || f + 8 > hend)) {  // leaves the last segment: look it up
            int m;
            const ss::PmEntry e = ss::lookup(mp, f, m);
            hkey = -1;
            if (f >= e.packed_off && f + 8 <= e.packed_off + e.len) {
                hkey = m;
                hend = e.packed_off + e.len;
                hdelta = e.param_off - e.packed_off;
                hslot = e.param - a.param_base;
            }
        }
        const int key = has ? hkey : -1, slot = hslot;
        const int64_t k = f + hdelta;  // index inside the parameter tensor
        const int key0 = __shfl_sync(kAll, key, 0);
        const bool uniform = __all_sync(kAll, !has || (key0 >= 0 && key == key0));
        uint4 p = make_uint4(0, 0, 0, 0);
        if (uniform) {
            const int nl = __popc(__ballot_sync(kAll, has));  // lanes 0..nl-1 hold vectors
            const int64_t k0 = __shfl_sync(kAll, k, 0);
            const int slot0 = __shfl_sync(kAll, slot, 0);
            // the lane's next vector, 8 rounds on: its state and (when it
            // stays in this segment) its first batch's gradient lines into L2
            // while this round computes, so the next round's copies wait for
            // L2 rather than DRAM
            auto prefetch_next = [&]() {
                const int64_t fn = f + kStride;
                if (it > 1 && fn < fend) {
                    ss::prefetch_l2(a.master + fn);
                    ss::prefetch_l2(a.exp_avg + fn);
                    ss::prefetch_l2(a.exp_avg_sq + fn);
                    if (fn + 8 <= hend) {
#pragma unroll
                        for (int r = 0; r < kStageBatch; ++r)
                            if (r < n)
                                ss::prefetch_l2(static_cast<const uint16_t*>(tab.p[r * a.w + slot0]) + fn +
                                                hdelta);
                    }
                }
            };
            float s[8];
            if (a.congruent) {  // one element offset H for every rank: a template constant
                const int h = (int)((reinterpret_cast<uintptr_t>(
                                         static_cast<const uint16_t*>(tab.p[slot0]) + k0) & 15u) >> 1);
                switch (h) {
                    case 0: staged_sum<NR, 0>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    case 1: staged_sum<NR, 1>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    case 2: staged_sum<NR, 2>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    case 3: staged_sum<NR, 3>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    case 4: staged_sum<NR, 4>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    case 5: staged_sum<NR, 5>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    case 6: staged_sum<NR, 6>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                    default: staged_sum<NR, 7>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next); break;
                }
            } else {
                staged_sum<NR, -1>(a, tab, slot0, k0, nl, lane, wst_s, wst, s, prefetch_next);
            }
            if (lane < nl) p = adam_vec(a, f, s, n, t0, t1, m0, m1, v0, v1);
        } else if (key >= 0) {  // a round that meets a segment end: this vector is inside one
            const uint16_t* g0 = static_cast<const uint16_t*>(tab.p[slot]) + k;
            const uint4 x = ss::ld_any16(g0);
            float s[8] = {ss::bf16_lo(x.x), ss::bf16_hi(x.x), ss::bf16_lo(x.y), ss::bf16_hi(x.y),
                          ss::bf16_lo(x.z), ss::bf16_hi(x.z), ss::bf16_lo(x.w), ss::bf16_hi(x.w)};
            for (int r = 1; r < n; ++r)
                add_rank(s, ss::ld_any16(static_cast<const uint16_t*>(tab.p[r * a.w + slot]) + k));
            p = adam_vec(a, f, s, n, t0, t1, m0, m1, v0, v1);
        } else if (has) {  // the vector meets a segment end: element by element
            if constexpr (NR > 0 && NR <= kMaxVec) {
                // the entry of element f + i: the last one starting at or before it
                int c;
                ss::PmEntry e = ss::lookup(mp, f, c);
                const float th[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
                const float mm[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
                const float vv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t x = f + i;
                    while (c + 1 < a.M && mp.pm[c + 1].packed_off <= x) e = mp.pm[++c];
                    if (x >= e.packed_off && x < e.packed_off + e.len)
                        step_elem<NR>(a, tab, e.param - a.param_base, x,
                                      e.param_off + (x - e.packed_off), th[i], mm[i], vv[i]);
                }
            } else {  // N > 8: one element at a time, with fewer registers
                for (int i = 0; i < 8; ++i) {
                    const int64_t x = f + i;
                    int c;
                    const ss::PmEntry ex = ss::lookup(mp, x, c);
                    if (x >= ex.packed_off && x < ex.packed_off + ex.len)
                        step_scalar<true>(a, tab, ex.param - a.param_base, x,
                                          ex.param_off + (x - ex.packed_off));
                }
            }
        }
        const int nkey = __shfl_down_sync(kAll, key, 1);
        const int pkey = __shfl_up_sync(kAll, key, 1);
        uint4 nx;
        nx.x = __shfl_down_sync(kAll, p.x, 1);
        nx.y = __shfl_down_sync(kAll, p.y, 1);
        nx.z = __shfl_down_sync(kAll, p.z, 1);
        nx.w = __shfl_down_sync(kAll, p.w, 1);
        if (key >= 0)
            store_outputs_lane(a, tab, goff, slot, k, p, nx, lane < 31 && nkey == key,
                               lane > 0 && pkey == key);
    }
    if (gw == nwarps && lane < 16) {
        const int i = lane;
        if (i < 8 ? i < ed.nh : i - 8 < ed.nt) {
            const int64_t x = i < 8 ? ed.h0 + i : ed.t0 + (i - 8);
            int c;
            const ss::PmEntry ex = ss::lookup(mp, x, c);
            if (x >= ex.packed_off && x < ex.packed_off + ex.len)
                step_scalar<true>(a, tab, ex.param - a.param_base, x, ex.param_off + (x - ex.packed_off));
        }
    }
    if (pdl & 2) asm volatile("griddepcontrol.wait;" ::: "memory");
}

using StagedKern = void (*)(const ss::PmEntry*, const int*, StagedRuns, int, int, StepArgs, PtrTab);

StagedKern pick_staged(int N, int* smem) {
    StagedKern k;
    switch (N) {
        case 1: k = fused_step_copyin_staged_kernel<1>; break;
        case 2: k = fused_step_copyin_staged_kernel<2>; break;
        case 3: k = fused_step_copyin_staged_kernel<3>; break;
        case 4: k = fused_step_copyin_staged_kernel<4>; break;
        case 5: k = fused_step_copyin_staged_kernel<5>; break;
        case 6: k = fused_step_copyin_staged_kernel<6>; break;
        case 7: k = fused_step_copyin_staged_kernel<7>; break;
        case 8: k = fused_step_copyin_staged_kernel<8>; break;
        // N = 16 unrolled: both rank batches known at compile time (0.89 -> 0.93
        // of measured on the 218M-param misaligned set)
        case 16: k = fused_step_copyin_staged_kernel<16>; break;
        default: k = fused_step_copyin_staged_kernel<0>; break;
    }
    *smem = N <= kStageBatch ? staged_smem_bytes(1) : staged_smem_bytes(0);
    return k;
}

// Opt the staged kernels into their shared memory (above the 48 KiB default
// for N > 8) and the largest shared-memory carveout, once per device.
int staged_prepare(StagedKern k, int smem) {
    static std::mutex mu;
    static std::vector<std::pair<int, StagedKern>> done;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return ss::cuda_fail(e);
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& d : done)
        if (d.first == dev && d.second == k) return SS_OK;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k),
                                 cudaFuncAttributePreferredSharedMemoryCarveout,
                                 (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return ss::cuda_fail(e);
    done.emplace_back(dev, k);
    return SS_OK;
}

using FlatAnyKern = void (*)(const ss::PmEntry*, const int*, int, int64_t, int64_t, EdgeElems,
                             StepArgs, PtrTab);

template <bool SMALL = false>
auto pick_flat_any(int N) {
    switch (N) {
        case 1: return fused_step_flat_any_kernel<1, SMALL>;
        case 2: return fused_step_flat_any_kernel<2, SMALL>;
        case 3: return fused_step_flat_any_kernel<3, SMALL>;
        case 4: return fused_step_flat_any_kernel<4, SMALL>;
        case 5: return fused_step_flat_any_kernel<5, SMALL>;
        case 6: return fused_step_flat_any_kernel<6, SMALL>;
        case 7: return fused_step_flat_any_kernel<7, SMALL>;
        case 8: return fused_step_flat_any_kernel<8, SMALL>;
        case 16: return fused_step_flat_any_kernel<16, SMALL>;
        default: return fused_step_flat_any_kernel<0, SMALL>;
    }
}

}  // namespace

extern "C" int fsdp_sharded_step(const ss_plan* plan, const ss_step* s, int group,
                                 ss_stream_t stream) {
    if (!plan || !s) return SS_EINVAL;
    if (!plan->has_dev) return SS_ENODEVICE;
    if (int drc = ss::check_device(plan)) return drc;
    if (plan->eb != 2) return SS_EINVAL;
    int64_t lo, hi;
    if (!ss::group_range(plan, group, &lo, &hi)) return SS_EINVAL;
    const int N = plan->N, n = plan->n;
    const bool unpacked = s->rank_param_grads != nullptr;
    if (unpacked == (s->rank_grads != nullptr)) return SS_EINVAL;  // exactly one gradient source
    if (!s->hp || !s->master || !s->exp_avg || !s->exp_avg_sq || !s->param_shards) return SS_EINVAL;
    const ss_adamw* hp = s->hp;
    if (hp->step < 1 || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) || !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) ||
        !(hp->eps >= 0.0) || !std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay))
        return SS_EINVAL;
    if (s->n_out < 0 || s->n_out > SS_MAX_REPLICAS || (s->n_out > 0 && !s->params_out))
        return SS_EINVAL;
    const void* bufs[5] = {s->master, s->exp_avg, s->exp_avg_sq, s->param_shards, s->reduced_grad_out};
    for (const void* b : bufs)
        if (b && !ss::aligned(b, 16)) return SS_EALIGN;
    const int pa = group < 0 ? 0 : plan->gfirst[group];
    const int pb = group < 0 ? n : plan->gfirst[group] + plan->gnp[group];
    StepArgs a;
    std::memset(&a, 0, sizeof a);
    if (!unpacked) {
        for (int r = 0; r < N; ++r) {
            if (!s->rank_grads[r] && hi > lo) return SS_EINVAL;
            if (!ss::aligned(s->rank_grads[r], 16)) return SS_EALIGN;
            a.packed_grads.p[r] = s->rank_grads[r];
        }
    }
    bool gen = !plan->vec_aligned;  // true: some run needs the general (realigning) kernel
    for (int i = pa; i < pb; ++i) {
        if (plan->numel[i] == 0) continue;
        for (int r = 0; unpacked && r < N; ++r) {
            const void* q = s->rank_param_grads[(size_t)r * n + i];
            if (!q) return SS_EINVAL;
            if (!ss::aligned(q, 2)) return SS_EALIGN;
            gen |= !ss::aligned(q, 16);
        }
        for (int j = 0; j < s->n_out; ++j) {
            const void* q = s->params_out[(size_t)j * n + i];
            if (!q) return SS_EINVAL;
            if (!ss::aligned(q, 2)) return SS_EALIGN;
            gen |= !ss::aligned(q, 16);
        }
    }
    a.master = s->master;
    a.exp_avg = s->exp_avg;
    a.exp_avg_sq = s->exp_avg_sq;
    a.shards = static_cast<uint16_t*>(s->param_shards);
    a.gout = s->reduced_grad_out;
    a.N = N;
    a.n_out = s->n_out;
    a.M = (int)plan->pm.size();
    a.c = make_coef(hp);
    const int per_param = (unpacked ? N : 0) + s->n_out;
    if (per_param > kTab) return SS_EINVAL;
    const int wmax = per_param > 0 ? kTab / per_param : (pb - pa > 0 ? pb - pa : 1);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    PtrTab tab;
    auto fill = [&](int wa, int wb) {
        a.param_base = wa;
        a.w = wb - wa;
        a.congruent = 1;
        // only the slots the kernels read: per_param per parameter of the window
        std::memset(&tab, 0, sizeof(void*) * (size_t)std::min(kTab, per_param * (wb - wa)));
        for (int i = wa; i < wb; ++i) {
            for (int r = 1; unpacked && r < N; ++r)
                if (plan->numel[i] > 0 &&
                    ((reinterpret_cast<uintptr_t>(s->rank_param_grads[(size_t)r * n + i]) ^
                      reinterpret_cast<uintptr_t>(s->rank_param_grads[i])) & 15u))
                    a.congruent = 0;
            for (int r = 0; unpacked && r < N; ++r)
                tab.p[r * a.w + (i - wa)] = const_cast<void*>(s->rank_param_grads[(size_t)r * n + i]);
            const int goff = unpacked ? N * a.w : 0;
            for (int j = 0; j < s->n_out; ++j)
                tab.p[goff + j * a.w + (i - wa)] = s->params_out[(size_t)j * n + i];
        }
    };
    bool staged_launched = false;  // a staged copy-in launch of this call is queued
    // The staged copy-in's runs of the current pointer table, launched
    // together by staged_flush: rounds of 32 vectors per warp, as many rounds
    // per warp as keep kCopyinMinWaves waves of CTAs over all the runs (at
    // most kCopyinIters), each run's CTAs after the last run's, and one extra
    // warp per run for its edge elements.  Launches after a call's first may
    // start while the one before ends (programmatic dependent launch); each
    // ends only after the one before it.
    StagedRuns staged;
    staged.n = 0;
    int64_t staged_vecs = 0;
    auto staged_flush = [&]() -> int {
        if (staged.n == 0) return SS_OK;
        int smem = 0;
        const StagedKern fk = pick_staged(N, &smem);
        int rc = staged_prepare(fk, smem);
        if (rc) return rc;
        const int64_t per_round = 32 * (int64_t)kStagedWarps;  // vectors per CTA round
        const int64_t it = staged_vecs / (per_round * kCopyinMinWaves * 3 * ss::num_sms());
        const int iters = (int)(it < 1 ? 1 : it > kCopyinIters ? kCopyinIters : it);
        const int64_t span = 32 * (int64_t)iters;  // vectors per warp
        staged.cta0[0] = 0;
        for (int i = 0; i < staged.n; ++i) {
            staged.nwarps[i] = (staged.nvec[i] + span - 1) / span;
            staged.cta0[i + 1] = staged.cta0[i] + (staged.nwarps[i] + 1 + kStagedWarps - 1) / kStagedWarps;
        }
        if (staged.cta0[staged.n] > 0x7FFFFFFF) return SS_EOVERFLOW;
        const int pdl = staged_launched ? 3 : 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)staged.cta0[staged.n]);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1] = {};
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = staged_launched ? 1 : 0;
        const cudaError_t le = cudaLaunchKernelEx(&cfg, fk, (const ss::PmEntry*)plan->d_pm,
                                                  (const int*)plan->d_pm_block, staged, iters, pdl, a, tab);
        rc = le == cudaSuccess ? ss::check_launch() : ss::cuda_fail(le);
        staged_launched = true;
        staged.n = 0;
        staged_vecs = 0;
        return rc;
    };
    // The step over packed range [rlo, rhi), whose data segments all belong to
    // the parameters in the pointer table.
    auto run = [&](int64_t rlo, int64_t rhi) -> int {
        if (rhi <= rlo) return SS_OK;
        if (!gen && rlo % 8 == 0 && rhi % 8 == 0) {
            // everything aligned: one thread per packed vector
            const int64_t nvec = (rhi - rlo) / 8;
            if (nvec <= kSmallVecs && per_param * a.w <= kTabSmall) {
                // a launch of a few waves: the small table, and programmatic
                // stream serialisation so that it may start while the grid
                // before it on the stream finishes
                PtrTabSmall ts;
                std::memcpy(ts.p, tab.p, sizeof ts.p);
                const auto fs = unpacked ? pick_flat<true, true>(N) : pick_flat<false, true>(N);
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3((unsigned)((nvec + kThreads - 1) / kThreads));
                cfg.blockDim = dim3(kThreads);
                cfg.stream = st;
                cudaLaunchAttribute attr[1] = {};
                attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
                attr[0].val.programmaticStreamSerializationAllowed = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                const cudaError_t le = cudaLaunchKernelEx(&cfg, fs, (const ss::PmEntry*)plan->d_pm,
                                                          (const int*)plan->d_pm_block, rlo, nvec, a, ts);
                return le == cudaSuccess ? ss::check_launch() : ss::cuda_fail(le);
            }
            FlatRoundsKern fr = unpacked && kFlatRounds > 0 ? pick_flat_rounds(N) : nullptr;
            if (fr) {
                // rounds of 32 vectors per warp, as many as keep kCopyinWaves
                // waves of CTAs (at most kFlatRounds)
                int64_t it = nvec / ((int64_t)kThreads * kCopyinWaves * 3 * ss::num_sms());
                const int iters = (int)(it < 1 ? 1 : it > kFlatRounds ? kFlatRounds : it);
                const int64_t span = 32 * (int64_t)iters;  // vectors per warp
                const int64_t nw = (nvec + span - 1) / span;
                constexpr int64_t kChunkW = (int64_t)1 << 32;  // warps per launch
                for (int64_t w0 = 0; w0 < nw; w0 += kChunkW) {
                    const int64_t cw = nw - w0 < kChunkW ? nw - w0 : kChunkW;
                    const int64_t cv = w0 + cw >= nw ? nvec - span * w0 : span * cw;
                    fr<<<(unsigned)((cw + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, st>>>(
                        plan->d_pm, plan->d_pm_block, rlo + 8 * span * w0, cv, iters, a, tab);
                    int rc = ss::check_launch();
                    if (rc) return rc;
                }
                return SS_OK;
            }
            FlatKern ff = unpacked ? pick_flat<true>(N) : pick_flat<false>(N);
            constexpr int64_t kMaxBlocks = 0x7FFFFFFF;
            for (int64_t v0 = 0; v0 < nvec; v0 += kMaxBlocks * kThreads) {
                const int64_t cnt = nvec - v0 < kMaxBlocks * kThreads ? nvec - v0 : kMaxBlocks * kThreads;
                ff<<<(unsigned)((cnt + kThreads - 1) / kThreads), kThreads, 0, st>>>(
                    plan->d_pm, plan->d_pm_block, rlo + 8 * v0, cnt, a, tab);
                int rc = ss::check_launch();
                if (rc) return rc;
            }
            return SS_OK;
        }
        // any alignment: per-lane realigned output stores; whole vectors
        // [lo8, hi8), the edges one by one
        const int64_t lo8 = (rlo + 7) / 8 * 8, hi8 = rhi / 8 * 8;
        EdgeElems ed;
        int64_t nvec = 0;
        if (lo8 <= hi8) {
            nvec = (hi8 - lo8) / 8;
            ed = EdgeElems{rlo, hi8, (int)(lo8 - rlo), (int)(rhi - hi8)};
        } else {  // the range lies inside one 8-element vector
            ed = EdgeElems{rlo, rhi, (int)(rhi - rlo), 0};
        }
        const EdgeElems none{0, 0, 0, 0};
        if (unpacked) {  // queued: one launch per pointer table (staged_flush)
            if (staged.n == kMaxRuns) {
                const int rc = staged_flush();
                if (rc) return rc;
            }
            const int i = staged.n++;
            staged.vbeg[i] = lo8;
            staged.nvec[i] = nvec;
            staged.ed[i] = ed;
            staged_vecs += nvec;
            return SS_OK;
        }
        if (nvec + 16 <= kSmallVecs && per_param * a.w <= kTabSmall) {
            // a launch of a few waves: the small table, and programmatic
            // stream serialisation (as for the aligned small form)
            PtrTabSmall ts;
            std::memcpy(ts.p, tab.p, sizeof ts.p);
            const auto fs = pick_flat_any<true>(N);
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)((nvec + 16 + kThreads - 1) / kThreads));
            cfg.blockDim = dim3(kThreads);
            cfg.stream = st;
            cudaLaunchAttribute attr[1] = {};
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            const cudaError_t le =
                cudaLaunchKernelEx(&cfg, fs, (const ss::PmEntry*)plan->d_pm, (const int*)plan->d_pm_block,
                                   (int)plan->pm.size(), lo8, nvec, ed, a, ts);
            return le == cudaSuccess ? ss::check_launch() : ss::cuda_fail(le);
        }
        FlatAnyKern ff = pick_flat_any(N);
        constexpr int64_t kChunk = (int64_t)0x7FFFFFF0 * kThreads;  // vectors per launch
        int64_t v0 = 0;
        do {
            const int64_t cnt = nvec - v0 < kChunk ? nvec - v0 : kChunk;
            const bool last = v0 + cnt >= nvec;
            const int64_t threads = cnt + (last ? 16 : 0);
            ff<<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(
                plan->d_pm, plan->d_pm_block, (int)plan->pm.size(), lo8 + 8 * v0, cnt,
                last ? ed : none, a, tab);
            int rc = ss::check_launch();
            if (rc) return rc;
            v0 += cnt;
        } while (v0 < nvec);
        return SS_OK;
    };
    if (hi <= lo || plan->pm.empty()) return SS_OK;
    if (pb - pa <= wmax) {  // one pointer table: the whole range at once
        fill(pa, pb);
        const int rc = run(lo, hi);
        return rc ? rc : staged_flush();
    }
    // More parameters than one pointer table: windows of consecutive
    // parameters, whole groups packed greedily into each (a group larger than
    // a window is cut into windows of its own).  In packed order a window's
    // data segments form runs broken only by segments of other parameters; a
    // window of whole groups is one run, since groups lie side by side, while
    // a cut group gives a run per rank shard.  Each run, pads included, is one
    // range.
    std::vector<std::pair<int, int>> windows;
    {
        const int ga = group < 0 ? 0 : group, gb = group < 0 ? plan->G : group + 1;
        int wa = pa, wb = pa;  // the window being filled: [wa, wb)
        for (int g = ga; g < gb; ++g) {
            const int g0 = plan->gfirst[g], g1 = g0 + plan->gnp[g];
            if (g1 - wa > wmax && wb > wa) {  // the group does not fit: close the window
                windows.emplace_back(wa, wb);
                wa = wb;
            }
            while (g1 - wa > wmax) {  // a group larger than a window
                windows.emplace_back(wa, wa + wmax);
                wa += wmax;
            }
            wb = g1;
        }
        if (wb > wa) windows.emplace_back(wa, wb);
    }
    const std::vector<ss::PmEntry>& pm = plan->pm;
    const size_t m0 = (size_t)(std::lower_bound(pm.begin(), pm.end(), lo,
                                                [](const ss::PmEntry& e, int64_t v) {
                                                    return e.packed_off < v;
                                                }) -
                               pm.begin());
    for (const auto& wnd : windows) {
        const int wa = wnd.first, wb = wnd.second;
        fill(wa, wb);
        int64_t rl = -1, rh = -1;
        for (size_t m = m0; m < pm.size() && pm[m].packed_off < hi; ++m) {
            if (pm[m].param >= wa && pm[m].param < wb) {
                if (rl < 0) rl = pm[m].packed_off;
                rh = pm[m].packed_off + pm[m].len;
            } else if (rl >= 0) {
                int rc = run(rl, rh);
                if (rc) return rc;
                rl = -1;
            }
        }
        if (rl >= 0) {
            int rc = run(rl, rh);
            if (rc) return rc;
        }
        int rc = staged_flush();  // before the next window refills the table
        if (rc) return rc;
    }
    return SS_OK;
}

