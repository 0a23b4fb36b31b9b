// linear_ce_small.cu -- linear cross entropy of a toy model in one launch.
//
// Where tokens, vocabulary and hidden size are all small, the chain of launches of
// linear_ce.cu is nothing but latency (five launches, 25 us, for 50 tokens, 128 x
// 64).  Here one cluster of 8 CTAs does it all: each takes an eighth of the
// vocabulary, with every token's hidden states and its own weight rows in shared
// memory as fp32.  The rows' statistics, and then the parts of dH, meet in one
// another's shared memory; P stays in fp32 registers and shared memory.
// CUDA-core products, 3 T V D fused multiply-adds over 8 SMs: 12.7 us at 50 x 128 x
// 64, most of it the latency of one step after another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "device_utils.cuh"
#include "internal.h"
#include "launch.cuh"

namespace {

using ss::launch_after;
using ss::wait_before;

constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kTokens = 64;           // most tokens
constexpr int kHidden = 256;          // and hidden size
constexpr int kSlice = 64;            // vocabulary rows of a CTA
constexpr int kLd = kTokens + 4;      // of the transposed arrays: 16-byte groups of 8 lanes fall in 32 banks
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    int T, D, V, per;  // per: vocabulary rows of a CTA
    const uint16_t* hidden;
    int64_t ldh;
    const uint16_t* weight;
    int64_t ldw;
    const int64_t* targets;
    int64_t ignore;
    int mean;
    float grad_scale;
    float* loss;
    float* token_loss;
    uint16_t* d_hidden;
    int64_t ld_dh;
    uint16_t* d_weight;
    int64_t ld_dw;
};

__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The word at `p`'s place in CTA `rank`'s shared memory.
__device__ __forceinline__ float peer(const float* p, int rank) {
    uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) ce_small_kernel(const Args a) {
    launch_after();
    extern __shared__ __align__(16) float mem[];
    const int D = a.D, ldw = D | 1;            // odd: a column of the weight slice has no bank conflicts
    float* ht = mem;                           // [D][kLd] hidden states, a token a column
    float* pt = ht + D * kLd;                  // [kSlice][kLd] logits, then P
    float* ws = pt + kSlice * kLd;             // [per][ldw]
    float* part = ws + ((a.per * ldw + 3) & ~3);  // [tokens][D] this slice's part of dH
    __shared__ int token[kTokens], target[kTokens], ignored[kTokens];
    __shared__ float top_s[kTokens], sum_s[kTokens], hit_s[kTokens];
    __shared__ float2 row_s[kTokens];  // log-sum-exp in base 2, the target's p - 1
    __shared__ float loss_s[kTokens];
    __shared__ int first;  // live tokens of the first 32
    const int rank = cluster_rank(), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int v0 = rank * a.per;
    const int rows = v0 >= a.V ? 0 : a.V - v0 < a.per ? a.V - v0 : a.per;

    wait_before();

    // the tokens that count, in order
    int64_t y = a.ignore;
    uint32_t mask = 0;
    if (warp < 2) {
        if (tid < a.T) y = a.targets[tid];
        mask = __ballot_sync(0xFFFFFFFFu, y != a.ignore);
        if (tid == 0) first = __popc(mask);
    }
    const int live = __syncthreads_count(warp < 2 && y != a.ignore);
    if (warp < 2) {
        const int at = (warp ? first : 0) + __popc(mask & ((1u << lane) - 1));
        if (y != a.ignore) {
            token[at] = tid;
            target[at] = y >= 0 && y < a.V ? (int)y : -1;
        } else if (tid < a.T && rank == 0 && a.token_loss) {
            a.token_loss[tid] = 0.f;
        }
    }
    if (warp < 2) ignored[tid] = y == a.ignore;
    constexpr int kWarps = kThreads / 32;
    for (int d = lane; d < D; d += 32) {
#pragma unroll 4
        for (int v = warp; v < rows; v += kWarps) ws[v * ldw + d] = ss::bf16_to_f32(a.weight[(v0 + v) * a.ldw + d]);
    }
    __syncthreads();
    const int quads = (live + 3) / 4;  // groups of 4 tokens
    for (int d = lane; d < D; d += 32) {
#pragma unroll 4
        for (int t = warp; t < 4 * quads; t += kWarps)
            ht[d * kLd + t] = t < live ? ss::bf16_to_f32(a.hidden[token[t] * a.ldh + d]) : 0.f;
    }
    if (a.d_hidden && rank == kCtas - 1) {
        for (int t = warp; t < a.T; t += kWarps)
            for (int d = lane; ignored[t] && d < D; d += 32) a.d_hidden[t * a.ld_dh + d] = 0;
    }
    __syncthreads();

    // logits: a thread a vocabulary row and 4 tokens
    for (int i = tid; i < quads * rows; i += kThreads) {
        const int t = 4 * (i / rows), v = i % rows;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < D; ++d) {
            const float w = ws[v * ldw + d];
            const float4 h = *reinterpret_cast<const float4*>(ht + d * kLd + t);
            s = make_float4(fmaf(w, h.x, s.x), fmaf(w, h.y, s.y), fmaf(w, h.z, s.z), fmaf(w, h.w, s.w));
        }
        *reinterpret_cast<float4*>(pt + v * kLd + t) = s;
    }
    __syncthreads();

    // the slice's maximum and sum of exponentials of a row, without the target's own
    for (int t = warp; t < live; t += kThreads / 32) {
        const int hit = target[t] - v0;
        float top = -INFINITY;
        for (int v = lane; v < rows; v += 32) top = v == hit ? top : fmaxf(top, pt[v * kLd + t]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float at = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        for (int v = lane; v < rows; v += 32) sum += v == hit ? 0.f : expf(pt[v * kLd + t] - at);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) {
            top_s[t] = top;
            sum_s[t] = sum;
            hit_s[t] = hit >= 0 && hit < rows ? pt[hit * kLd + t] : -INFINITY;
        }
    }
    cluster_sync();
    if (tid < live) {
        float top = -INFINITY, sum = 0.f, hit = -INFINITY, m[kCtas], s[kCtas];
#pragma unroll
        for (int r = 0; r < kCtas; ++r) {
            m[r] = peer(top_s + tid, r), s[r] = peer(sum_s + tid, r);
            const float x = peer(hit_s + tid, r);
            hit = x == -INFINITY ? hit : x;  // one slice holds it; a NaN comes through
            top = fmaxf(top, m[r]);
        }
        const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int r = 0; r < kCtas; ++r) sum += m[r] == -INFINITY ? s[r] : s[r] * expf(m[r] - at);
        if (target[tid] < 0) hit = NAN;
        // with r the other classes' mass over the target's: loss = log(1 + r), p - 1 = -r / (1 + r)
        float d = top == -INFINITY && sum == 0.f ? -INFINITY : (at - hit) + logf(sum);
        // no loss without a target's logit, with one of +inf (inf - inf), or with nothing but -inf
        if (!(hit < INFINITY) || (hit == -INFINITY && d == -INFINITY)) d = NAN;
        const float rest = expf(-fabsf(d));
        const float l = (d > 0.f ? d : 0.f) + log1pf(rest);
        // of a target at -inf the loss is infinite, and log-sum-exp what the other classes have
        const float lse = hit == -INFINITY ? at + logf(sum) : hit + l;
        row_s[tid] = make_float2(lse * kLog2e, -(d > 0.f ? 1.f : rest) / (1.f + rest));
        loss_s[tid] = l;
        if (rank == 0 && a.token_loss) a.token_loss[token[tid]] = l;
    }
    __syncthreads();
    if (rank == 0 && warp == 0) {
        double s = 0.0;
        for (int t = lane; t < live; t += 32) s += (double)loss_s[t];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_down_sync(0xFFFFFFFFu, s, d);
        if (lane == 0) *a.loss = (float)(a.mean && live > 0 ? s / live : s);
    }
    if (a.d_hidden || a.d_weight) {
        const float scale = a.mean ? (live > 0 ? a.grad_scale / (float)live : 0.f) : a.grad_scale;
        for (int t = lane; t < 4 * quads; t += 32) {
            const float2 r = t < live ? row_s[t] : make_float2(0.f, 0.f);
            const int hit = t < live ? target[t] - v0 : -1;
            for (int v = warp; v < rows; v += kWarps) {
                float* p = pt + v * kLd + t;
                *p = t >= live ? 0.f : v == hit ? r.y : exp2f(fmaf(*p, kLog2e, -r.x));
            }
        }
        __syncthreads();
        if (a.d_weight) {  // a thread a column and 4 vocabulary rows
            const int groups = (rows + 3) / 4;
            for (int i = tid; i < groups * D; i += kThreads) {
                const int d = i % D, v = 4 * (i / D);
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                for (int t = 0; t < 4 * quads; t += 4) {
                    const float4 h = *reinterpret_cast<const float4*>(ht + d * kLd + t);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 p = *reinterpret_cast<const float4*>(pt + (v + k) * kLd + t);
                        if (v + k < rows)
                            s[k] = fmaf(p.x, h.x, fmaf(p.y, h.y, fmaf(p.z, h.z, fmaf(p.w, h.w, s[k]))));
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (v + k < rows) a.d_weight[(v0 + v + k) * a.ld_dw + d] = ss::f32_to_bf16(scale * s[k]);
            }
        }
        if (a.d_hidden) {
            for (int i = tid; i < quads * D; i += kThreads) {
                const int d = i % D, t = 4 * (i / D);
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int v = 0; v < rows; ++v) {
                    const float w = ws[v * ldw + d];
                    const float4 p = *reinterpret_cast<const float4*>(pt + v * kLd + t);
                    s = make_float4(fmaf(w, p.x, s.x), fmaf(w, p.y, s.y), fmaf(w, p.z, s.z), fmaf(w, p.w, s.w));
                }
                part[t * D + d] = s.x, part[(t + 1) * D + d] = s.y;
                part[(t + 2) * D + d] = s.z, part[(t + 3) * D + d] = s.w;
            }
            cluster_sync();
            for (int t = rank + kCtas * warp; t < live; t += kCtas * (kThreads / 32)) {
                for (int d = lane; d < D; d += 32) {
                    float s = 0.f;
#pragma unroll
                    for (int r = 0; r < kCtas; ++r) s += peer(part + t * D + d, r);
                    a.d_hidden[token[t] * a.ld_dh + d] = ss::f32_to_bf16(scale * s);
                }
            }
        }
    }
    cluster_sync();  // nobody leaves while its shared memory may still be read
}

int smem_bytes(int D, int per) {
    return 4 * (D * kLd + kSlice * kLd + ((per * (D | 1) + 3) & ~3) + kTokens * D);
}

constexpr int kMaxSmem = 4 * (kHidden * kLd + kSlice * kLd + kSlice * (kHidden + 1) + kTokens * kHidden);
static_assert(kMaxSmem <= 222 * 1024, "the largest sizes fit an SM");

}  // namespace

namespace ss {

// Time of a training call, here and by the launches of linear_ce.cu, as measured side by
// side when the rule was chosen (tokens x vocabulary x hidden size): 50 x 128 x 64 13.9 (12.7
// by now) and 24.9 us, 64 x 256 x 64 17.1 and
// 25.2, 8 x 512 x 256 22.3 and 27.4, 64 x 64 x 256 28.0 and 27.8; with twice the work
// those are ahead (64 x 300 x 128 30.9 and 27.2), and without gradients everywhere.
bool linear_ce_fits_small(int64_t T, int64_t D, int64_t V) {
    return T >= 1 && T <= kTokens && D <= kHidden && V <= kCtas * kSlice && T * D * V <= kSmallWork;
}

int linear_ce_small(const ss_linear_ce* p, cudaStream_t st) {
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(ce_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
    }
    Args a = {};
    a.T = (int)p->num_tokens, a.D = (int)p->hidden_size, a.V = (int)p->vocab_size;
    a.per = (a.V + kCtas - 1) / kCtas;
    a.hidden = static_cast<const uint16_t*>(p->hidden), a.ldh = p->hidden_stride;
    a.weight = static_cast<const uint16_t*>(p->weight), a.ldw = p->weight_stride;
    a.targets = p->targets, a.ignore = p->ignore_index;
    a.mean = p->reduction == SS_LOSS_MEAN, a.grad_scale = (float)p->grad_scale;
    a.loss = p->loss_out, a.token_loss = p->token_loss_out;
    a.d_hidden = static_cast<uint16_t*>(p->d_hidden), a.ld_dh = p->d_hidden_stride;
    a.d_weight = static_cast<uint16_t*>(p->d_weight), a.ld_dw = p->d_weight_stride;
    return launch(ce_small_kernel, kCtas, kThreads, smem_bytes(a.D, a.per), 0, true, st, a);
}

}  // namespace ss
