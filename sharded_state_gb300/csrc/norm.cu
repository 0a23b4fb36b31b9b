// norm.cu -- dropout, and the residual stream's step between two layers: dropout of
// the branch, the residual's addition and the root-mean-square norm, with the
// backward pass.
//
//   h  = round(dropout(x) + residual)      the stream, in its type
//   r  = 1 / sqrt(mean_c h_c^2 + eps)      one per row, fp32
//   y  = h r w                             rounded to the type, or to MXFP8
//
//   n  = h r,  g = dy w
//   dh = r (g - n mean_c(g n)) + d_sum     d_sum: what arrives at h from elsewhere
//   dx = dropout(dh)                       the same mask, made again
//   dw = sum over the rows of dy n
//
// The statistics are taken of h as it is stored, so that the backward pass, which
// reads the stored h, is the gradient of what the forward pass computed.
//
// Each element moves once, and the memory is what bounds it: a row stays in its threads'
// registers (8 elements a load, up to 8 loads a thread) between the sum over it and the
// outputs.  16384 x 4096 bf16, 537 MB either way: forward 81 us (6.6 TB/s, where a copy
// makes 6.8), backward with d_weight 93 us (5.8 TB/s; 169 us without the next row on its
// way).  With dropout the generator's instructions come on top: 100 us and, with d_x
// written too, 119; by itself, 8192 x 11008, dropout takes 67 us, 5.4 TB/s, two thirds of
// the issue slots.  Four and eight loads a thread, of more than 8192 columns, spill
// registers (all but the forward pass of bf16 rows on 16 bytes or of four loads, and of
// fp32 rows of four on 16 bytes): 2000 x 16384 bf16 forward 58, backward 102 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "philox.cuh"
#include "tcgen05.cuh"
#include "vec8.cuh"

namespace {

namespace tc = ss::tc;

using ss::launch_after;
using ss::Run;
using ss::Vec8;
using ss::wait_before;

// ---------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------

constexpr int kDropThreads = 256;

struct DropArgs {
    int64_t rows;
    int groups, last;  // groups of 8 columns in a row, columns of the last one
    const void* x;
    int64_t x_stride;
    void* out;
    int64_t out_stride;
    const int64_t* rng;
    uint32_t drop;
    float scale;
    int64_t step_rows;  // the grid's threads (or warps), as rows and groups (or pieces)
    int step_groups;
    int64_t x_step, out_step;  // and as elements
};

// A warp takes pieces of kDropPiece groups of a row, two a lane: a place in the matrix is
// worked out once for both, and both are on their way before the first is worked on (8192
// x 11008: 72.5 -> 66.8 us).
constexpr int kDropPiece = 64;

template <class T, bool ALIGNED>
__global__ void __launch_bounds__(kDropThreads) dropout_rows_kernel(const __grid_constant__ DropArgs a) {
    launch_after();
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const int pieces = (a.groups + kDropPiece - 1) / kDropPiece;
    const int64_t first = (int64_t)blockIdx.x * (kDropThreads / 32) + warp;
    int64_t row = first / pieces;
    int piece = (int)(first - row * pieces);
    wait_before();
    const ss::Philox philox(a.rng);
    for (; row < a.rows; row += a.step_rows) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        T* out = static_cast<T*>(a.out) + row * a.out_stride;
        const int g0 = piece * kDropPiece + lane;
        Vec8<T> v[2];
        uint4 tail[2] = {};
        auto run = [&](int g) {  // of the columns from this group on, as far as two groups go
            return Run(g + 2 < a.groups ? 16 : (a.groups - 1 - g) * 8 + a.last, lane == 0, lane == 31);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = g0 + 32 * i;
            v[i].template fetch<ALIGNED>(x + 8 * (int64_t)g, run(g), tail[i]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int g = g0 + 32 * i;
            v[i].template settle<ALIGNED>(x + 8 * (int64_t)g, run(g), tail[i]);
            float f[8];
            v[i].get(f);
            ss::drop8(f, philox((uint32_t)row, (uint32_t)g), a.drop, a.scale);
            v[i].set(f);
            v[i].template store<ALIGNED>(out + 8 * (int64_t)g, run(g));
        }
        piece += a.step_groups;
        if (piece >= pieces) piece -= pieces, ++row;
    }
}

// Narrow matrices, whose rows would leave lanes of such pieces idle: threads take groups of
// 8 in the order of the matrix, as far apart as the grid has
// threads; places in it are carried on by adding (with a row's index times its stride for
// each group it was 181 instructions a group for 145).
template <class T, bool ALIGNED>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropArgs a) {
    launch_after();
    const int64_t first = (int64_t)blockIdx.x * kDropThreads + threadIdx.x;
    const int lane = threadIdx.x & 31;
    int64_t row = first / a.groups;
    int group = (int)(first - row * a.groups);
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + 8 * (int64_t)group;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + 8 * (int64_t)group;
    const int64_t x_turn = a.x_stride - 8 * (int64_t)a.groups, out_turn = a.out_stride - 8 * (int64_t)a.groups;
    wait_before();
    const ss::Philox philox(a.rng);
    while (ALIGNED ? row < a.rows : __any_sync(0xFFFFFFFFu, row < a.rows)) {
        const int after = group + 2 < a.groups ? 8 : group + 1 < a.groups ? a.last : 0;  // columns of the next group
        const Run run(row >= a.rows ? 0 : after ? 8 + after : a.last, lane == 0 || group == 0, lane == 31);
        Vec8<T> v;
        v.template load<ALIGNED>(x, run);
        float f[8];
        v.get(f);
        ss::drop8(f, philox((uint32_t)row, (uint32_t)group), a.drop, a.scale);
        v.set(f);
        v.template store<ALIGNED>(out, run);
        row += a.step_rows;
        group += a.step_groups;
        x += a.x_step;
        out += a.out_step;
        if (group >= a.groups) group -= a.groups, ++row, x += x_turn, out += out_turn;
    }
}

// ---------------------------------------------------------------------------
// the norm
// ---------------------------------------------------------------------------

struct NormArgs {
    int64_t rows;
    int cols, team;  // team: threads of a row
    const void *x, *residual, *weight;
    int64_t x_stride, residual_stride;
    float eps, inv_cols;
    const int64_t* rng;
    uint32_t drop;
    float scale;
    void *sum_out, *out;
    int64_t sum_stride, out_stride;
    float* rstd_out;
    unsigned char *mx_data, *mx_scales;
    int mx_tiles;  // tiles of 128 columns
};

struct NormGradArgs {
    int64_t rows;
    int cols, team;
    const void *d_out, *h, *weight, *d_sum;
    int64_t d_out_stride, h_stride, d_sum_stride;
    const float* rstd;
    float inv_cols;
    const int64_t* rng;
    uint32_t drop;
    float scale;
    void *d_h, *d_x;
    int64_t d_h_stride, d_x_stride;
    float* part;     // [gridDim.x][cols]: each CTA's share of d_weight, to be joined by another kernel
    void* d_weight;  // or: the grid is one cluster that joins them itself
};

// Sum over a row's team, the same in all of its threads: over the warp in registers,
// then over the warps in a fixed order through `lane_sums` (one float a warp; another
// one at every other call).
__device__ __forceinline__ float team_sum(float s, int team, float* lane_sums) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
    if (team == 32) return s;
    const int warp = threadIdx.x >> 5, warps = team >> 5, first = warp / warps * warps;
    if ((threadIdx.x & 31) == 0) lane_sums[warp] = s;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < warps; ++i) t += lane_sums[first + i];
    return t;
}

__device__ __forceinline__ void store_weight(uint16_t* p, float v) { *p = ss::f32_to_bf16(v); }
__device__ __forceinline__ void store_weight(float* p, float v) { *p = v; }

// 8 normed values as MXFP8: their block is this lane's and its 3 neighbours'.
__device__ __forceinline__ void store_mx8(const NormArgs& a, int64_t row, int col, const float (&y)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, ss::abs_bits(y[i]));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (row >= a.rows || col >= a.mx_tiles * ss::kMxTile) return;
    const uint32_t byte = ss::mx_scale<SS_MXFP8>(top);
    const float inverse = ss::mx_inverse(byte);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = byte == 255u ? 0.f : y[i] * inverse;
    *reinterpret_cast<uint2*>(a.mx_data + (row * a.mx_tiles * ss::kMxTile + col)) = ss::Mx<SS_MXFP8>::encode(f);
    if ((threadIdx.x & 3) == 0) a.mx_scales[ss::mx_scale_at(row, col >> 5, a.mx_tiles)] = (unsigned char)byte;
}

// Most threads of a row, for one, two and more loads a thread; two or three rows of 512 fit
// an SM's registers.  At any alignment a load holds a block more, and where 512 threads
// would take four loads each, one row an SM: more threads of fewer loads (1801 x 9589,
// forward 86 -> 68 us, backward 141 -> 86; 13018 x 5155 backward in one load of 672 threads
// 353, two of 352 446; forward in one 330, in two 236; 2000 x 6001 fp32 forward in one load
// of 768 63, two of 384 66).
constexpr int kMostThreads = 512;
constexpr int norm_threads(int vecs, bool aligned, int elem_bytes) {
    return aligned || vecs * elem_bytes != 4 ? kMostThreads : elem_bytes == 2 ? 768 : 1024;
}
constexpr int grad_threads(int vecs, bool aligned, int elem_bytes) {
    return aligned || elem_bytes > 2 || vecs > 2 ? kMostThreads : vecs == 1 ? 768 : 640;
}

// Rows of more than 256 threads and two loads of bf16 each are held to 56 registers, so
// that three rows of 352 threads fit an SM (8192 x 5632 with dropout, forward: 76 us, where
// 58 registers and two rows take 91).
template <class T, int VECS, bool ALIGNED>
constexpr bool three_rows() { return ALIGNED && VECS <= 2 && sizeof(T) == 2; }

// VECS loads of 8 elements a thread, `team` threads a row, blockDim / team rows a CTA.
// WIDE: of more than 256 threads.
template <class T, int VECS, bool ALIGNED, bool WIDE>
__global__ void __launch_bounds__(!WIDE ? 256 : three_rows<T, VECS, ALIGNED>() ? 576 : norm_threads(VECS, ALIGNED, sizeof(T)),
                                  WIDE && three_rows<T, VECS, ALIGNED>() ? 2 : 0)
norm_kernel(const __grid_constant__ NormArgs a) {
    constexpr bool kWeightAhead = VECS <= 4;  // asked for with the row
    __shared__ float lane_sums[32];
    launch_after();
    const int mine = threadIdx.x % a.team, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / a.team) + threadIdx.x / a.team;
    const bool live = row < a.rows;
    auto run = [&](int col) { return Run(live ? a.cols - col : 0, lane == 0, lane == 31); };
    wait_before();
    Vec8<T> x[VECS], r[VECS], w[VECS];
    uint4 x_tail[VECS] = {}, r_tail[VECS] = {}, w_tail[VECS] = {};
    const T* x_row = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r_row = static_cast<const T*>(a.residual) + row * a.residual_stride;
    const T* weight = static_cast<const T*>(a.weight);
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int col = 8 * (mine + i * a.team);
        x[i].template fetch<ALIGNED>(x_row + col, run(col), x_tail[i]);
        if (a.residual) r[i].template fetch<ALIGNED>(r_row + col, run(col), r_tail[i]);
    }
    if (kWeightAhead) {
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int col = 8 * (mine + i * a.team);
            w[i].template fetch<ALIGNED>(weight + col, run(col), w_tail[i]);
        }
    }
    ss::Philox philox;
    if (a.drop) philox = ss::Philox(a.rng);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int col = 8 * (mine + i * a.team);
        float f[8];
        x[i].template settle<ALIGNED>(x_row + col, run(col), x_tail[i]);
        if (a.drop || a.residual) {
            x[i].get(f);
            if (a.drop) ss::drop8(f, philox((uint32_t)row, (uint32_t)(col >> 3)), a.drop, a.scale);
            if (a.residual) {
                float q[8];
                r[i].template settle<ALIGNED>(r_row + col, run(col), r_tail[i]);
                r[i].get(q);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = __fadd_rn(f[k], q[k]);
            }
            x[i].set(f);
        }
        if (a.sum_out) x[i].template store<ALIGNED>(static_cast<T*>(a.sum_out) + row * a.sum_stride + col, run(col));
        x[i].get(f);  // zeros behind the row's end
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(f[k], f[k], s);
    }
    s = team_sum(s, a.team, lane_sums);
    const float rstd = 1.f / sqrtf(fmaf(s, a.inv_cols, a.eps));
    if (live && mine == 0 && a.rstd_out) a.rstd_out[row] = rstd;
    if (!a.out && !a.mx_data) return;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int col = 8 * (mine + i * a.team);
        if (!kWeightAhead) w[i].template fetch<ALIGNED>(weight + col, run(col), w_tail[i]);
        w[i].template settle<ALIGNED>(weight + col, run(col), w_tail[i]);
        float f[8], q[8];
        x[i].get(f);
        w[i].get(q);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * rstd * q[k];
        if (a.out) {
            w[i].set(f);
            w[i].template store<ALIGNED>(static_cast<T*>(a.out) + row * a.out_stride + col, run(col));
        }
        if (a.mx_data) {
            const int n = run(col).n;  // an infinite rstd would make the zeros behind the end NaN
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = k < n ? f[k] : 0.f;
            store_mx8(a, row, col, f);
        }
    }
}

constexpr int kCluster = 8;  // CTAs of a backward pass that joins d_weight itself, at the most

// The rows of a backward pass in turn, each CTA its own; the next row's elements are
// on their way while one is worked on, where the registers hold both.
template <class T, int VECS, bool ALIGNED>
__host__ __device__ constexpr bool loads_ahead() { return VECS * sizeof(T) <= (ALIGNED ? 4 : 2) || VECS == 1; }

// Rows too long for the registers are read twice, the second time from L2: those of eight
// loads a thread, but for aligned ones of bf16 (backward of 1000 x 20000, held 92 us and
// read twice 136; of 1000 x 20001 772 and 231, of 500 x 32768 fp32 278 and 99: what is
// held there spills; of four loads, 1801 x 9589 held 140 and read twice 179).
template <class T, int VECS, bool ALIGNED>
__host__ __device__ constexpr bool holds_row() { return VECS < 8 || (ALIGNED && sizeof(T) == 2); }

template <class T, int VECS, bool ALIGNED, bool WIDE>
__global__ void __launch_bounds__(WIDE ? grad_threads(VECS, ALIGNED, sizeof(T)) : kMostThreads)
norm_grad_kernel(const __grid_constant__ NormGradArgs a) {
    extern __shared__ float joined[];  // [rows at a time][cols], where that is more than one
    __shared__ float lane_sums[2][32];
    constexpr bool kAhead = !WIDE && loads_ahead<T, VECS, ALIGNED>(), kHold = holds_row<T, VECS, ALIGNED>();
    constexpr int kHeld = kHold ? VECS : 1;
    launch_after();
    const int mine = threadIdx.x % a.team, teams = blockDim.x / a.team, team = threadIdx.x / a.team;
    const int lane = threadIdx.x & 31;
    wait_before();
    float dw[VECS][8];
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[i][k] = 0.f;
    auto run = [&](int64_t row, int col) { return Run(row < a.rows ? a.cols - col : 0, lane == 0, lane == 31); };
    struct Row {
        Vec8<T> dy[kHeld], h[kHeld], ds[kHeld];
        uint4 dy_tail[kHeld], h_tail[kHeld], ds_tail[kHeld];
        float rstd;
    };
    // Loads i of a row, or one of them, into place `to`.
    auto fetch_one = [&](Row& x, int to, int64_t row, int i) {
        const int col = 8 * (mine + i * a.team);
        x.dy_tail[to] = x.h_tail[to] = x.ds_tail[to] = make_uint4(0, 0, 0, 0);
        x.dy[to].template fetch<ALIGNED>(static_cast<const T*>(a.d_out) + row * a.d_out_stride + col, run(row, col), x.dy_tail[to]);
        x.h[to].template fetch<ALIGNED>(static_cast<const T*>(a.h) + row * a.h_stride + col, run(row, col), x.h_tail[to]);
        x.ds[to].clear();
        if (a.d_sum)
            x.ds[to].template fetch<ALIGNED>(static_cast<const T*>(a.d_sum) + row * a.d_sum_stride + col, run(row, col), x.ds_tail[to]);
    };
    auto settle_one = [&](Row& x, int to, int64_t row, int i) {
        const int col = 8 * (mine + i * a.team);
        x.dy[to].template settle<ALIGNED>(static_cast<const T*>(a.d_out) + row * a.d_out_stride + col, run(row, col), x.dy_tail[to]);
        x.h[to].template settle<ALIGNED>(static_cast<const T*>(a.h) + row * a.h_stride + col, run(row, col), x.h_tail[to]);
        if (a.d_sum)
            x.ds[to].template settle<ALIGNED>(static_cast<const T*>(a.d_sum) + row * a.d_sum_stride + col, run(row, col), x.ds_tail[to]);
    };
    auto fetch = [&](Row& x, int64_t row) {
        if (kHold) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) fetch_one(x, kHold ? i : 0, row, i);
        }
        x.rstd = row < a.rows ? a.rstd[row] : 0.f;
    };
    auto settle = [&](Row& x, int64_t row) {
        if (kHold) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) settle_one(x, kHold ? i : 0, row, i);
        }
    };
    // The place of loads i of a row that may have to be read again.
    auto place = [&](Row& x, int64_t row, int i) {
        if (kHold) return i;
        fetch_one(x, 0, row, i);
        settle_one(x, 0, row, i);
        return 0;
    };
    int parity = 0;
    const int64_t step = (int64_t)gridDim.x * teams;
    Row x, ahead;
    Vec8<T> w[kAhead ? VECS : 1];
    if (kAhead) {
        fetch(x, (int64_t)blockIdx.x * teams + team);
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int col = 8 * (mine + i * a.team);
            w[i].template load<ALIGNED>(static_cast<const T*>(a.weight) + col, Run(a.cols - col, lane == 0, lane == 31));
        }
    }
    ss::Philox philox;
    if (a.drop && a.d_x) philox = ss::Philox(a.rng);
    auto weight = [&](int i, float (&g)[8]) {
        if (!kAhead) {
            const int col = 8 * (mine + i * a.team);
            w[0].template load<ALIGNED>(static_cast<const T*>(a.weight) + col, Run(a.cols - col, lane == 0, lane == 31));
        }
        w[kAhead ? i : 0].get(g);
    };
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += step, parity ^= 1) {
        const int64_t row = first + team;
        if (kAhead)
            fetch(ahead, row + step);
        else
            fetch(x, row);
        settle(x, row);
        const float rstd = x.rstd;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            float f[8], q[8], g[8];
            const int at = place(x, row, i);
            weight(i, g);
            x.dy[at].get(f);
            x.h[at].get(q);
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // zeros behind the row's end
                const float t = f[k] * (q[k] * rstd);
                s = fmaf(t, g[k], s);
                dw[i][k] += t;
            }
        }
        s = team_sum(s, a.team, lane_sums[parity]) * a.inv_cols;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int col = 8 * (mine + i * a.team);
            float f[8], q[8], g[8], d[8];
            const int at = place(x, row, i);
            weight(i, g);
            x.dy[at].get(f);
            x.h[at].get(q);
            x.ds[at].get(d);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = fmaf(rstd, fmaf(-q[k] * rstd, s, f[k] * g[k]), d[k]);
            Vec8<T> v;
            if (a.d_h) {
                v.set(f);
                v.template store<ALIGNED>(static_cast<T*>(a.d_h) + row * a.d_h_stride + col, run(row, col));
            }
            if (a.d_x) {
                if (a.drop) ss::drop8(f, philox((uint32_t)row, (uint32_t)(col >> 3)), a.drop, a.scale);
                v.set(f);
                v.template store<ALIGNED>(static_cast<T*>(a.d_x) + row * a.d_x_stride + col, run(row, col));
            }
        }
        if (kAhead) x = ahead;
    }
    if (!a.part && !a.d_weight) return;
    float* part = a.part + (int64_t)blockIdx.x * a.cols;
    float* to = teams > 1 || a.d_weight ? joined + team * a.cols : part;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int col = 8 * (mine + i * a.team);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (col + k < a.cols) to[col + k] = dw[i][k];
    }
    if (to == part) return;
    __syncthreads();
    float* joint = a.d_weight ? joined : part;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float s = 0.f;
        for (int t = 0; t < teams; ++t) s += joined[t * a.cols + c];
        joint[c] = s;
    }
    if (!a.d_weight) return;
    tc::cluster_sync();
    const int ctas = gridDim.x, share = (a.cols + ctas - 1) / ctas, c0 = blockIdx.x * share;
    for (int c = c0 + threadIdx.x; c < min(c0 + share, a.cols); c += blockDim.x) {
        float v[kCluster], s = 0.f;
#pragma unroll
        for (int q = 0; q < kCluster; ++q) {
            v[q] = 0.f;
            if (q < ctas)
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[q]) : "r"(tc::map_to_rank(tc::smem_addr(joined + c), q)));
        }
#pragma unroll
        for (int q = 0; q < kCluster; ++q) s += v[q];
        store_weight(static_cast<T*>(a.d_weight) + c, s);
    }
    tc::cluster_sync();
}

// d_weight: the CTAs' shares summed in a fixed order, 32 columns a CTA.
constexpr int kJoinRows = 16;

template <class T>
__global__ void __launch_bounds__(32 * kJoinRows) norm_join_kernel(const float* part, int parts, int cols, T* out) {
    __shared__ float sums[kJoinRows][33];
    launch_after();
    wait_before();
    const int lane = threadIdx.x & 31, line = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (col < cols) {
#pragma unroll 8
        for (int p = line; p < parts; p += kJoinRows) s += part[(int64_t)p * cols + col];
    }
    sums[line][lane] = s;
    __syncthreads();
    if (line > 0 || col >= cols) return;
#pragma unroll
    for (int i = 1; i < kJoinRows; ++i) s += sums[i][lane];
    store_weight(out + col, s);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxCols = 32768;  // 512 threads hold a row, 8 loads each
constexpr int64_t kMaxFlat = (int64_t)1 << 33;  // columns of dropout: groups count in 32 bits

// Threads of a row and of a CTA, and loads of 8 elements a thread.
struct Shape {
    int vecs, team, threads;
};

// `most` loads a thread (1 or 2) as long as that many threads may take a row, then as few
// as do.  Two, 2048 x 2048 forward: 8.2 us where one takes 9.1 and four 9.7.
template <class F>
Shape choose_shape(int64_t vectors, int most, F&& most_threads) {
    int team = 32;
    while (team < 256 && team * most < vectors) team *= 2;
    if (team * most >= vectors) return {vectors <= team ? 1 : 2, team, 256};
    int vecs = most;
    while (vecs * most_threads(vecs) < vectors) vecs *= 2;
    team = (int)((vectors + vecs - 1) / vecs + 31) / 32 * 32;
    return {vecs, team, team};
}

// The forward pass's, and the backward pass's: one load a thread for unaligned rows (1021
// x 1001 forward: 6.9 -> 6.3 us), and where fp32 rows would leave the backward pass no
// registers for the next row's.
Shape choose_norm_shape(int64_t vectors, int elem_bytes, bool aligned) {
    return choose_shape(vectors, aligned ? 2 : 1, [&](int vecs) { return norm_threads(vecs, aligned, elem_bytes); });
}
Shape choose_grad_shape(int64_t cols, int elem_bytes, bool aligned) {
    return choose_shape((cols + 7) / 8, elem_bytes == 2 && aligned ? 2 : 1,
                        [&](int vecs) { return grad_threads(vecs, aligned, elem_bytes); });
}

// CTAs that take the rows of a backward pass in turn, as many as the registers hold.
int64_t grad_grid(int64_t rows, const Shape& s) {
    const int64_t teams = s.threads / s.team, need = (rows + teams - 1) / teams;
    return std::min(need, (int64_t)ss::num_sms() * (s.threads > 256 ? 1 : 2));
}

template <class F>
int with_shape(int elem_bytes, int vecs, bool aligned, F&& f) {
    auto pick = [&](auto t, auto v) { return aligned ? f(t, v, std::true_type()) : f(t, v, std::false_type()); };
    auto vec = [&](auto t) {
        switch (vecs) {
            case 1: return pick(t, std::integral_constant<int, 1>());
            case 2: return pick(t, std::integral_constant<int, 2>());
            case 4: return pick(t, std::integral_constant<int, 4>());
            default: return pick(t, std::integral_constant<int, 8>());
        }
    };
    return elem_bytes == 2 ? vec(uint16_t()) : vec(float());
}

// A matrix that may be absent: its row stride, its addresses.
struct Matrix {
    const void* p;
    int64_t stride;
};

int check_matrices(int64_t rows, int64_t cols, int elem_bytes, std::initializer_list<Matrix> list) {
    for (const Matrix& m : list) {
        if (!m.p) continue;
        if (m.stride < cols) return SS_EINVAL;
        if (rows > 0 && m.stride > INT64_MAX / 8 / rows) return SS_EOVERFLOW;
    }
    for (const Matrix& m : list)
        if (!ss::aligned(m.p, (uintptr_t)elem_bytes)) return SS_EALIGN;
    return SS_OK;
}

// Rows of all of them on 16 bytes.
bool rows_on_16(int elem_bytes, std::initializer_list<Matrix> list) {
    for (const Matrix& m : list)
        if (m.p && (!ss::aligned(m.p, 16) || m.stride * elem_bytes % 16 != 0)) return false;
    return true;
}

// A probability in steps of 2^-16 and the factor of what is kept; SS_EINVAL where
// nothing would be.
int choose_drop(double p, const int64_t* rng, uint32_t* drop, float* scale) {
    if (!(p >= 0.0 && p < 1.0)) return SS_EINVAL;
    *drop = (uint32_t)std::nearbyint(p * 65536.0);
    if (*drop >= 65536u) return SS_EINVAL;
    if (*drop > 0 && !rng) return SS_EINVAL;
    *scale = (float)(65536.0 / (65536.0 - *drop));
    return ss::aligned(rng, 8) ? SS_OK : SS_EALIGN;
}

}  // namespace

extern "C" {

int ss_dropout(int64_t rows, int64_t cols, int elem_bytes, const void* x, int64_t x_stride, void* out,
               int64_t out_stride, double p, const int64_t* rng, ss_stream_t stream) {
    if (rows < 0 || cols < 0 || (elem_bytes != 2 && elem_bytes != 4)) return SS_EINVAL;
    DropArgs a = {};
    if (int rc = choose_drop(p, rng, &a.drop, &a.scale)) return rc;
    if (!rng) return SS_EINVAL;
    if (rows == 0 || cols == 0) return SS_OK;
    if (!x || !out) return SS_EINVAL;
    if (rows > kMaxRows || cols > kMaxFlat) return SS_EOVERFLOW;
    if (int rc = check_matrices(rows, cols, elem_bytes, {{x, x_stride}, {out, out_stride}})) return rc;
    a.rows = rows, a.groups = (int)((cols + 7) / 8), a.last = (int)(cols - 8 * (int64_t)(a.groups - 1));
    a.x = x, a.x_stride = x_stride, a.out = out, a.out_stride = out_stride, a.rng = rng;
    const int64_t total = a.rows * a.groups;
    const int64_t grid = std::min((total + kDropThreads - 1) / kDropThreads, (int64_t)ss::num_sms() * 8);
    const bool al = rows_on_16(elem_bytes, {{x, x_stride}, {out, out_stride}});
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t pieces = (a.groups + kDropPiece - 1) / kDropPiece;
    if (4 * (int64_t)a.groups >= 3 * kDropPiece * pieces) {  // three lanes of four have work
        constexpr int64_t kWarps = kDropThreads / 32;
        const int64_t ctas = std::min((a.rows * pieces + kWarps - 1) / kWarps, (int64_t)ss::num_sms() * 8);
        a.step_rows = ctas * kWarps / pieces;
        a.step_groups = (int)(ctas * kWarps % pieces);
        const auto kernel = elem_bytes == 2 ? (al ? dropout_rows_kernel<uint16_t, true> : dropout_rows_kernel<uint16_t, false>)
                                            : (al ? dropout_rows_kernel<float, true> : dropout_rows_kernel<float, false>);
        return ss::launch(kernel, ctas, kDropThreads, 0, 0, true, st, a);
    }
    a.step_rows = grid * kDropThreads / a.groups;
    a.step_groups = (int)(grid * kDropThreads % a.groups);
    a.x_step = a.step_rows * x_stride + 8 * (int64_t)a.step_groups;
    a.out_step = a.step_rows * out_stride + 8 * (int64_t)a.step_groups;
    const auto kernel = elem_bytes == 2 ? (al ? dropout_kernel<uint16_t, true> : dropout_kernel<uint16_t, false>)
                                        : (al ? dropout_kernel<float, true> : dropout_kernel<float, false>);
    return ss::launch(kernel, grid, kDropThreads, 0, 0, true, st, a);
}

int ss_rms_norm(const ss_norm* n, ss_stream_t stream) {
    if (!n || n->rows < 0 || n->cols < 1 || (n->elem_bytes != 2 && n->elem_bytes != 4)) return SS_EINVAL;
    if (!(n->eps >= 0.0) || !std::isfinite((float)n->eps)) return SS_EINVAL;
    NormArgs a = {};
    if (int rc = choose_drop(n->dropout, n->rng, &a.drop, &a.scale)) return rc;
    if (n->rows > kMaxRows || n->cols > kMaxCols) return SS_EOVERFLOW;
    if (n->rows == 0) return SS_OK;
    if (!n->sum_out && !n->out && !n->rstd_out && !n->mx_data) return SS_EINVAL;
    if (!n->x || !n->weight || !n->mx_data != !n->mx_scales) return SS_EINVAL;
    const Matrix x = {n->x, n->x_stride}, res = {n->residual, n->residual_stride}, w = {n->weight, n->cols};
    const Matrix sum = {n->sum_out, n->sum_stride}, out = {n->out, n->out_stride};
    if (int rc = check_matrices(n->rows, n->cols, n->elem_bytes, {x, res, w, sum, out})) return rc;
    if (!ss::aligned(n->rstd_out, 4) || !ss::aligned(n->mx_data, 16) || !ss::aligned(n->mx_scales, 16)) return SS_EALIGN;
    a.rows = n->rows, a.cols = (int)n->cols;
    a.x = n->x, a.x_stride = n->x_stride, a.residual = n->residual, a.residual_stride = n->residual_stride;
    a.weight = n->weight, a.eps = (float)n->eps, a.inv_cols = 1.f / (float)n->cols, a.rng = n->rng;
    a.sum_out = n->sum_out, a.sum_stride = n->sum_stride, a.out = n->out, a.out_stride = n->out_stride;
    a.rstd_out = n->rstd_out;
    a.mx_data = static_cast<unsigned char*>(n->mx_data), a.mx_scales = static_cast<unsigned char*>(n->mx_scales);
    a.mx_tiles = (int)((n->cols + ss::kMxTile - 1) / ss::kMxTile);
    // the weight is one row: its own stride does not matter
    const bool al = rows_on_16(n->elem_bytes, {x, res, sum, out}) && ss::aligned(n->weight, 16);
    const Shape s = choose_norm_shape(n->mx_data ? (int64_t)a.mx_tiles * (ss::kMxTile / 8) : (n->cols + 7) / 8, n->elem_bytes, al);
    a.team = s.team;
    const int64_t teams = s.threads / s.team, grid = (n->rows + teams - 1) / teams;
    return with_shape(n->elem_bytes, s.vecs, al, [&](auto t, auto v, auto aligned) {
        constexpr int V = decltype(v)::value;
        constexpr bool A = decltype(aligned)::value;
        // what choose_norm_shape gives: of unaligned fp32 rows one load by up to 1024 threads, then four
        constexpr bool kNarrow = V == 1 || (V == 2 && A), kWide = V > 1 || !A, kNever = V == 2 && !A && sizeof(t) == 4;
        if constexpr (kNever) {
            return SS_EINVAL;
        } else {
            const auto kernel = s.threads > 256 ? norm_kernel<decltype(t), V, A, kWide> : norm_kernel<decltype(t), V, A, !kNarrow>;
            return ss::launch(kernel, grid, s.threads, 0, 0, true, reinterpret_cast<cudaStream_t>(stream), a);
        }
    });
}

int ss_rms_norm_workspace(int64_t rows, int64_t cols, size_t* bytes_out) {
    if (rows < 0 || cols < 1 || !bytes_out) return SS_EINVAL;
    if (rows > kMaxRows || cols > kMaxCols) return SS_EOVERFLOW;
    *bytes_out = (size_t)(std::max<int64_t>(std::min(rows, (int64_t)ss::num_sms() * 2), 1) * cols * 4);
    return SS_OK;
}

int ss_rms_norm_backward(const ss_norm_grad* n, ss_stream_t stream) {
    if (!n || n->rows < 0 || n->cols < 1 || (n->elem_bytes != 2 && n->elem_bytes != 4)) return SS_EINVAL;
    if (n->rows > 0 && !n->d_h && !n->d_x && !n->d_weight) return SS_EINVAL;
    NormGradArgs a = {};
    if (int rc = choose_drop(n->dropout, n->rng, &a.drop, &a.scale)) return rc;
    if (n->rows > kMaxRows || n->cols > kMaxCols) return SS_EOVERFLOW;
    if (!n->weight || (n->rows > 0 && (!n->d_out || !n->h || !n->rstd))) return SS_EINVAL;
    const Matrix dy = {n->d_out, n->d_out_stride}, h = {n->h, n->h_stride}, ds = {n->d_sum, n->d_sum_stride};
    const Matrix w = {n->weight, n->cols}, dh = {n->d_h, n->d_h_stride}, dx = {n->d_x, n->d_x_stride};
    if (int rc = check_matrices(n->rows, n->cols, n->elem_bytes, {dy, h, ds, w, dh, dx, {n->d_weight, n->cols}}))
        return rc;
    if (!ss::aligned(n->rstd, 4) || !ss::aligned(n->workspace, 16)) return SS_EALIGN;
    size_t wanted = 0;
    if (int rc = ss_rms_norm_workspace(n->rows, n->cols, &wanted)) return rc;
    if (n->d_weight && (!n->workspace || n->workspace_bytes < wanted)) return SS_EINVAL;
    const bool al = rows_on_16(n->elem_bytes, {dy, h, ds, dh, dx}) && ss::aligned(n->weight, 16);
    const Shape s = choose_grad_shape(n->cols, n->elem_bytes, al);
    int64_t grid = std::max<int64_t>(grad_grid(n->rows, s), 1);
    if (n->rows == 0 && !n->d_weight) return SS_OK;
    a.rows = n->rows, a.cols = (int)n->cols, a.team = s.team;
    a.d_out = n->d_out, a.d_out_stride = n->d_out_stride, a.h = n->h, a.h_stride = n->h_stride;
    a.weight = n->weight, a.d_sum = n->d_sum, a.d_sum_stride = n->d_sum_stride, a.rstd = n->rstd;
    a.inv_cols = 1.f / (float)n->cols, a.rng = n->rng;
    a.d_h = n->d_h, a.d_h_stride = n->d_h_stride, a.d_x = n->d_x, a.d_x_stride = n->d_x_stride;
    const int teams = s.threads / s.team;
    // Few rows, one for each team of 8 CTAs, are one cluster's, which joins d_weight in its
    // shared memory: one launch for two (50 x 64, calls back to back: 12.5 -> 8.0 us).  With
    // rows in turn the two launches are as short or shorter (32 x 4096 in a graph: 9.1 us in
    // a cluster, 6.2 in two launches), and with four loads a thread even for one row (1 x
    // 8976: 14.4, 9.5).
    const bool cluster = n->d_weight && s.vecs <= 2 && teams * a.cols * 4 <= 48 * 1024 - 512 && n->rows <= kCluster * teams;
    if (cluster) {
        grid = std::min<int64_t>((n->rows + teams - 1) / teams, kCluster);
        grid = std::max<int64_t>(grid, 1);
        a.d_weight = n->d_weight;
    } else if (n->d_weight) {
        a.part = static_cast<float*>(n->workspace);
    }
    // with several teams at most 8 x 512 floats, 4 x 1024 or 2 x 2048
    const int smem = teams > 1 || cluster ? teams * a.cols * 4 : 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (int rc = with_shape(n->elem_bytes, s.vecs, al, [&](auto t, auto v, auto aligned) {
            using T = decltype(t);
            constexpr int V = decltype(v)::value;
            constexpr bool A = decltype(aligned)::value;
            const auto kernel = s.threads > kMostThreads
                                    ? norm_grad_kernel<T, V, A, (grad_threads(V, A, sizeof(T)) > kMostThreads)>
                                    : norm_grad_kernel<T, V, A, false>;
            return ss::launch(kernel, grid, s.threads, smem, cluster ? (int)grid : 0, true, st, a);
        }))
        return rc;
    if (cluster) return SS_OK;
    if (!n->d_weight) return SS_OK;
    const int64_t blocks = (n->cols + 31) / 32;
    if (n->elem_bytes == 2)
        return ss::launch(norm_join_kernel<uint16_t>, blocks, 32 * kJoinRows, 0, 0, true, st, a.part, (int)grid, a.cols,
                          static_cast<uint16_t*>(n->d_weight));
    return ss::launch(norm_join_kernel<float>, blocks, 32 * kJoinRows, 0, 0, true, st, a.part, (int)grid, a.cols,
                      static_cast<float*>(n->d_weight));
}

}  // extern "C"
