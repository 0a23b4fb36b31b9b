// mx_quantize.cu -- matrices to microscaled floats and back (formats and layout:
// mx.cuh).
//
// A CTA takes 128 x 128 elements, which are one tile of scales whichever way the
// blocks run.  The blocks along the rows are formed on the way in, by 4 neighbouring
// lanes; for the transpose the tile is kept in shared memory and each thread takes
// two columns of 32 rows.  So one read of the matrix serves both, and the memory is
// what bounds it: 2 bytes read and 0.53 (MXFP4) or 1.03 (MXFP8) written for each
// element and orientation.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "philox.cuh"
#include "tma_host.h"
#include "vec8.cuh"

namespace {

using ss::kMxTile;
using ss::launch_after;
using ss::Mx;
using ss::Run;
using ss::Vec8;
using ss::wait_before;

constexpr int kThreads = 256;
constexpr int kRounds = kMxTile * kMxTile / 8 / kThreads;  // loads of 8 elements a thread

struct QuantArgs {
    int64_t rows, cols;
    int64_t row_tiles, col_tiles;
    const void* x;
    int64_t stride;
    unsigned char *data, *scales, *t_data, *t_scales;
    const int64_t* rng;
};

// Element as the format's, in units of the scale: exact where RANDOM, else left to
// the conversion's rounding.
template <int FORMAT, bool RANDOM>
__device__ __forceinline__ float element(float x, uint32_t byte, float inverse, uint32_t bits) {
    if (byte == 255u) return 0.f;
    const float v = x * inverse;
    return RANDOM ? ss::mx_round_random<FORMAT>(v, (float)bits * 0x1p-16f) : v;
}

template <class T, bool RANDOM>
constexpr int tile_bytes() {
    return kMxTile * kMxTile * (int)(sizeof(T) + (RANDOM ? 2 : 0));
}

template <class T, int FORMAT, bool TRANSPOSE, bool RANDOM, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ QuantArgs a) {
    using M = Mx<FORMAT>;
    using Word = typename M::Word;
    extern __shared__ __align__(16) unsigned char raw[];
    T* tile = reinterpret_cast<T*>(raw);                                        // [128][128]
    uint16_t* random = reinterpret_cast<uint16_t*>(raw + kMxTile * kMxTile * sizeof(T));  // [128][128]
    launch_after();
    const int64_t tr = blockIdx.x / a.col_tiles, tc = blockIdx.x - tr * a.col_tiles;
    const int line = threadIdx.x >> 4, c8 = threadIdx.x & 15;
    const int64_t row0 = tr * kMxTile, col0 = tc * kMxTile;
    wait_before();
    const T* x = static_cast<const T*>(a.x) + row0 * a.stride + col0 + 8 * c8;
    Vec8<T> v[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int r = 16 * i + line;
        v[i].template load<ALIGNED>(x + r * a.stride,
                                    Run(row0 + r < a.rows ? a.cols - col0 - 8 * c8 : 0, c8 == 0, c8 == 15));
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int r = 16 * i + line;
        const int64_t row = row0 + r;
        if (!TRANSPOSE && row - (line & 1) >= a.rows) break;  // both rows of the warp are behind the last
        uint4 bits = make_uint4(0, 0, 0, 0);
        if (RANDOM) bits = ss::Philox(a.rng)((uint32_t)row, (uint32_t)(tc * 16 + c8));
        if (TRANSPOSE) {
            v[i].template store<true>(tile + r * kMxTile + 8 * c8, Run(8, true, true));
            if (RANDOM) *reinterpret_cast<uint4*>(random + r * kMxTile + 8 * c8) = bits;
        }
        if (!a.data) continue;
        float f[8];
        v[i].get(f);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, ss::abs_bits(f[k]));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t byte = ss::mx_scale<FORMAT>(top);
        const float inverse = ss::mx_inverse(byte);
        const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = element<FORMAT, RANDOM>(f[k], byte, inverse, w[k >> 1] >> (16 * (k & 1)) & 0xFFFFu);
        // the row's 4 scales of the tile in its first lane
        uint32_t four = byte << (8 * (c8 >> 2));
        four |= __shfl_xor_sync(0xFFFFFFFFu, four, 4);
        four |= __shfl_xor_sync(0xFFFFFFFFu, four, 8);
        if (row < a.rows) {
            unsigned char* out = a.data + (row * a.col_tiles + tc) * M::kTileRow + c8 * (int)sizeof(Word);
            *reinterpret_cast<Word*>(out) = M::encode(f);
            if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(a.scales + ss::mx_scale_at(row, 4 * tc, a.col_tiles)) = four;
        }
    }
    if (!TRANSPOSE) return;
    __syncthreads();
    const int pair = threadIdx.x & 63, block = threadIdx.x >> 6;
    float f[2][kMxTile / 4];
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const T* at = tile + (32 * block + k) * kMxTile + 2 * pair;
        if (sizeof(T) == 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(at);
            f[0][k] = ss::bf16_lo(w), f[1][k] = ss::bf16_hi(w);
        } else {
            const float2 w = *reinterpret_cast<const float2*>(at);
            f[0][k] = w.x, f[1][k] = w.y;
        }
        top[0] = max(top[0], ss::abs_bits(f[0][k]));
        top[1] = max(top[1], ss::abs_bits(f[1][k]));
    }
    uint32_t byte[2];
    float inverse[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) byte[j] = ss::mx_scale<FORMAT>(top[j]), inverse[j] = ss::mx_inverse(byte[j]);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        uint32_t u = 0;
        if (RANDOM) u = *reinterpret_cast<const uint32_t*>(random + (32 * block + k) * kMxTile + 2 * pair);
        f[0][k] = element<FORMAT, RANDOM>(f[0][k], byte[0], inverse[0], u & 0xFFFFu);
        f[1][k] = element<FORMAT, RANDOM>(f[1][k], byte[1], inverse[1], u >> 16);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t row = col0 + 2 * pair + j;  // of the transpose
        if (row >= a.cols) break;
        unsigned char* out = a.t_data + (row * a.row_tiles + tr) * M::kTileRow + block * (M::kTileRow / 4);
        __align__(16) uint32_t words[M::kTileRow / 16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float g[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = f[j][8 * i + k];
            *reinterpret_cast<Word*>(words + i * (int)sizeof(Word) / 4) = M::encode(g);
        }
#pragma unroll
        for (int i = 0; i < M::kTileRow / 64; ++i)
            *reinterpret_cast<uint4*>(out + 16 * i) =
                make_uint4(words[4 * i], words[4 * i + 1], words[4 * i + 2], words[4 * i + 3]);
        a.t_scales[ss::mx_scale_at(row, 4 * tr + block, a.row_tiles)] = (unsigned char)byte[j];
    }
}

struct DequantArgs {
    int64_t rows, cols, col_tiles;
    const unsigned char *data, *scales;
    void* out;
    int64_t stride;
};

template <class T, int FORMAT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ DequantArgs a) {
    using M = Mx<FORMAT>;
    using Word = typename M::Word;
    launch_after();
    const int64_t tr = blockIdx.x / a.col_tiles, tc = blockIdx.x - tr * a.col_tiles;
    const int line = threadIdx.x >> 4, c8 = threadIdx.x & 15;
    const int64_t col = tc * kMxTile + 8 * c8;
    wait_before();
    Word w[kRounds];
    unsigned char byte[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int64_t row = tr * kMxTile + 16 * i + line;
        w[i] = Word();
        byte[i] = 0;
        if (row >= a.rows || col >= a.cols) continue;
        w[i] = *reinterpret_cast<const Word*>(a.data + (row * a.col_tiles + tc) * M::kTileRow + c8 * (int)sizeof(Word));
        byte[i] = a.scales[ss::mx_scale_at(row, col >> 5, a.col_tiles)];
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int64_t row = tr * kMxTile + 16 * i + line;
        if (row - (line & 1) >= a.rows) break;  // both rows of the warp are behind the last
        float f[8];
        M::decode(w[i], f);
        const float scale = ss::mx_value(byte[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= scale;
        Vec8<T> v;
        v.set(f);
        v.template store<ALIGNED>(static_cast<T*>(a.out) + row * a.stride + col,
                                  Run(row < a.rows ? a.cols - col : 0, c8 == 0, c8 == 15));
    }
}

constexpr int64_t kMaxSize = INT32_MAX;

int64_t tiles(int64_t n) { return (n + kMxTile - 1) / kMxTile; }

bool valid_format(int format) { return format == SS_MXFP4 || format == SS_MXFP8; }

// f of two truth values as types.
template <class F>
int with_flags(bool first, bool second, F&& f) {
    auto with_second = [&](auto x) { return second ? f(x, std::true_type()) : f(x, std::false_type()); };
    return first ? with_second(std::true_type()) : with_second(std::false_type());
}

template <class T, int FORMAT>
int launch_quantize(const QuantArgs& a, bool transpose, bool random, bool aligned, cudaStream_t st) {
    const int64_t grid = a.row_tiles * a.col_tiles;
    return with_flags(transpose, random, [&](auto t, auto r) {
        constexpr bool TR = decltype(t)::value, RA = decltype(r)::value;
        static std::atomic<uint64_t> ready[2]{};
        const int smem = TR ? tile_bytes<T, RA>() : 0;
        const auto kernel = aligned ? quantize_kernel<T, FORMAT, TR, RA, true> : quantize_kernel<T, FORMAT, TR, RA, false>;
        if (smem > 48 * 1024)
            if (int rc = ss::allow_smem(ready[aligned], reinterpret_cast<const void*>(kernel), smem)) return rc;
        return ss::launch(kernel, grid, kThreads, smem, 0, true, st, a);
    });
}

}  // namespace

extern "C" {

int ss_mx_bytes(int64_t rows, int64_t cols, int format, size_t* data_bytes, size_t* scale_bytes) {
    if (rows < 0 || cols < 0 || !valid_format(format) || !data_bytes || !scale_bytes) return SS_EINVAL;
    if (rows > kMaxSize || cols > kMaxSize) return SS_EOVERFLOW;
    *data_bytes = (size_t)rows * (size_t)tiles(cols) * (format == SS_MXFP4 ? 64 : 128);
    *scale_bytes = (size_t)tiles(rows) * (size_t)tiles(cols) * ss::kMxTileBytes;
    return SS_OK;
}

int ss_mx_quantize(const ss_mx_quant* q, ss_stream_t stream) {
    if (!q || q->rows < 0 || q->cols < 0 || !valid_format(q->format) || (q->elem_bytes != 2 && q->elem_bytes != 4))
        return SS_EINVAL;
    if (q->rows > kMaxSize || q->cols > kMaxSize) return SS_EOVERFLOW;
    if (q->rows == 0 || q->cols == 0) return SS_OK;
    if (!q->data != !q->scales || !q->t_data != !q->t_scales || (!q->data && !q->t_data)) return SS_EINVAL;
    if (!q->x || q->stride < q->cols) return SS_EINVAL;
    if (q->stride > INT64_MAX / 8 / q->rows || tiles(q->rows) * tiles(q->cols) > INT32_MAX) return SS_EOVERFLOW;
    if (!ss::aligned(q->x, (uintptr_t)q->elem_bytes) || !ss::aligned(q->data, 16) || !ss::aligned(q->scales, 16) ||
        !ss::aligned(q->t_data, 16) || !ss::aligned(q->t_scales, 16) || !ss::aligned(q->rng, 8))
        return SS_EALIGN;
    const QuantArgs a = {q->rows, q->cols, tiles(q->rows), tiles(q->cols), q->x, q->stride,
                         static_cast<unsigned char*>(q->data), static_cast<unsigned char*>(q->scales),
                         static_cast<unsigned char*>(q->t_data), static_cast<unsigned char*>(q->t_scales), q->rng};
    const bool aligned = ss::aligned(q->x, 16) && q->stride * q->elem_bytes % 16 == 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool t = q->t_data, r = q->rng;
    if (q->format == SS_MXFP4)
        return q->elem_bytes == 2 ? launch_quantize<uint16_t, SS_MXFP4>(a, t, r, aligned, st)
                                  : launch_quantize<float, SS_MXFP4>(a, t, r, aligned, st);
    return q->elem_bytes == 2 ? launch_quantize<uint16_t, SS_MXFP8>(a, t, r, aligned, st)
                              : launch_quantize<float, SS_MXFP8>(a, t, r, aligned, st);
}

int ss_mx_dequantize(int64_t rows, int64_t cols, int format, const void* data, const void* scales, void* out,
                     int64_t out_stride, int elem_bytes, ss_stream_t stream) {
    if (rows < 0 || cols < 0 || !valid_format(format) || (elem_bytes != 2 && elem_bytes != 4)) return SS_EINVAL;
    if (rows > kMaxSize || cols > kMaxSize) return SS_EOVERFLOW;
    if (rows == 0 || cols == 0) return SS_OK;
    if (!data || !scales || !out || out_stride < cols) return SS_EINVAL;
    if (out_stride > INT64_MAX / 8 / rows || tiles(rows) * tiles(cols) > INT32_MAX) return SS_EOVERFLOW;
    if (!ss::aligned(out, (uintptr_t)elem_bytes) || !ss::aligned(data, 16) || !ss::aligned(scales, 16)) return SS_EALIGN;
    const DequantArgs a = {rows, cols, tiles(cols), static_cast<const unsigned char*>(data),
                           static_cast<const unsigned char*>(scales), out, out_stride};
    const bool aligned = ss::aligned(out, 16) && out_stride * elem_bytes % 16 == 0;
    return with_flags(format == SS_MXFP4, elem_bytes == 4, [&](auto four, auto wide) {
        constexpr int F = decltype(four)::value ? SS_MXFP4 : SS_MXFP8;
        using T = std::conditional_t<decltype(wide)::value, float, uint16_t>;
        return ss::launch(aligned ? dequantize_kernel<T, F, true> : dequantize_kernel<T, F, false>,
                          tiles(rows) * a.col_tiles, kThreads, 0, 0, true, reinterpret_cast<cudaStream_t>(stream), a);
    });
}

}  // extern "C"
