// mx_quantize.cu -- matrices to microscaled floats and back (formats and layout:
// mx.cuh).
//
// A CTA takes 64 rows of 128 columns, half a tile of scales whichever way the blocks
// run.  The blocks along the rows are formed on the way in, by 4 neighbouring lanes; for
// the transpose the elements are kept in shared memory and each thread takes two columns
// of 32 rows.  So one read of the matrix serves both: 2 bytes read and 0.53
// (MXFP4) or 1.03 (MXFP8) written for each element and orientation.
//
// To the nearest along the rows the memory bounds it (32000 x 2048 bf16 to MXFP4: 28 us,
// 6.0 TB/s; back 26 us, 6.4 TB/s).  Both ways nothing is full (18 instructions an element
// on 65 % of the issue slots, the integer pipe 61 %; 8192 x 2048 12.4 us, 4.1 TB/s).  At
// random it is 41 instructions an element both ways, the integer pipe busy three quarters
// of the time (8192 x 5632 65 us, of which the generator is 15, rounding at random rather
// than to the nearest 22).
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "launch.cuh"
#include "mx.cuh"
#include "philox.cuh"
#include "vec8.cuh"

namespace {

using ss::kMxTile;
using ss::launch_after;
using ss::Mx;
using ss::Run;
using ss::Vec8;
using ss::wait_before;

constexpr int kThreads = 128;
constexpr int kLines = kThreads / 16;  // rows loaded at a time: 16 lanes take 128 columns
constexpr int kRounds = 8;             // loads of 8 elements a thread
constexpr int kFewRounds = 2;          // without the transpose, where 64 rows a CTA would leave SMs idle
constexpr int kRows = kLines * kRounds, kBlocks = kRows / 32;

struct QuantArgs {
    int64_t rows, cols;
    int64_t row_tiles, col_tiles;
    const void* x;
    int64_t stride;
    unsigned char *data, *scales, *t_data, *t_scales;
    const int64_t* rng;
};

template <class T, bool RANDOM>
constexpr int tile_bytes() {
    return kRows * kMxTile * (int)(sizeof(T) + (RANDOM ? 2 : 0));
}

// Bits of the largest magnitude of 8 elements.
__device__ __forceinline__ uint32_t largest(const Vec8<uint16_t>& v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.r.x & 0x7FFF7FFFu, v.r.y & 0x7FFF7FFFu),
                                __vmaxu2(v.r.z & 0x7FFF7FFFu, v.r.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t largest(const Vec8<float>& v) {
    float f[8];
    v.get(f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, ss::abs_bits(f[i]));
    return m;
}

template <int FORMAT, bool RANDOM>
__device__ __forceinline__ typename Mx<FORMAT>::Word encode(const float (&f)[8], uint32_t byte, const uint32_t (&u)[8]) {
    if (byte == 255u) return typename Mx<FORMAT>::Word();
    return RANDOM ? ss::mx_encode_random<FORMAT>(f, ss::mx_inverse(byte), u)
                  : ss::mx_encode<FORMAT>(f, ss::mx_inverse(byte));
}

// Rows of a tile in shared memory, in words, those of every 32 rows turned by 16 words
// more: threads that read 16 neighbouring pairs of columns of 2 blocks of rows at once
// meet all banks.
template <int WORDS>
__device__ __forceinline__ int turned(int row, int word) {
    return row * WORDS + ((word + 16 * (row >> 5)) & (WORDS - 1));
}

// Two columns of 32 rows out of the tile, as two's 16-bit halves or as floats.
template <class T>
struct Columns;

template <>
struct Columns<uint16_t> {
    uint32_t w[32];
    __device__ __forceinline__ void load(const uint32_t* tile, int block, int pair) {
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = tile[turned<kMxTile / 2>(32 * block + k, pair)];
    }
    __device__ __forceinline__ void largest(uint32_t (&top)[2]) const {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
        top[0] = m << 16, top[1] = m & 0xFFFF0000u;
    }
    __device__ __forceinline__ float get(int j, int k) const { return j ? ss::bf16_hi(w[k]) : ss::bf16_lo(w[k]); }
};

template <>
struct Columns<float> {
    float w[32][2];
    __device__ __forceinline__ void load(const uint32_t* tile, int block, int pair) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const float2 v = *reinterpret_cast<const float2*>(tile + turned<kMxTile>(32 * block + k, 2 * pair));
            w[k][0] = v.x, w[k][1] = v.y;
        }
    }
    __device__ __forceinline__ void largest(uint32_t (&top)[2]) const {
        top[0] = top[1] = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            top[0] = max(top[0], ss::abs_bits(w[k][0]));
            top[1] = max(top[1], ss::abs_bits(w[k][1]));
        }
    }
    __device__ __forceinline__ float get(int j, int k) const { return w[k][j]; }
};

// ROUNDS x 8 rows of 128 columns: kRows for the transpose.
template <class T, int FORMAT, int ROUNDS, bool TRANSPOSE, bool RANDOM, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && ALIGNED ? (RANDOM ? 5 : 6) : 4) quantize_kernel(const __grid_constant__ QuantArgs a) {
    using M = Mx<FORMAT>;
    using Word = typename M::Word;
    constexpr int kWords = kMxTile * (int)sizeof(T) / 4;  // of a row of the tile
    extern __shared__ __align__(16) uint32_t tile[];      // [kRows][kWords], then the random bits, [kRows][64]
    uint32_t* random = tile + kRows * kWords;
    launch_after();
    const int64_t part = blockIdx.x / a.col_tiles, tc = blockIdx.x - part * a.col_tiles;
    const int64_t row0 = part * (kLines * ROUNDS), col0 = tc * kMxTile;
    const int line = threadIdx.x >> 4, c8 = threadIdx.x & 15;
    wait_before();
    const T* x = static_cast<const T*>(a.x) + (row0 + line) * a.stride + col0 + 8 * c8;
    const int rows = (int)min(a.rows - row0, (int64_t)(kLines * ROUNDS)), left = (int)min(a.cols - col0 - 8 * c8, (int64_t)16);
    Vec8<T> v[ROUNDS];
    uint4 tail[ROUNDS] = {};
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i)
        v[i].template fetch<ALIGNED>(x + kLines * i * a.stride, Run(kLines * i + line < rows ? left : 0, c8 == 0, c8 == 15), tail[i]);
    const int64_t pitch = a.col_tiles * M::kTileRow;
    unsigned char* out = a.data + (row0 + line) * pitch + tc * M::kTileRow + c8 * (int)sizeof(Word);
    unsigned char* scales = a.scales + ss::mx_scale_at(row0, 4 * tc, a.col_tiles) + 16 * line;
    const ss::Philox philox = RANDOM ? ss::Philox(a.rng) : ss::Philox();
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i, out += kLines * pitch) {
        const int r = kLines * i + line;
        if (!TRANSPOSE && kLines * i + (line & ~1) >= rows) break;  // both rows of the warp are behind the last
        v[i].template settle<ALIGNED>(x + kLines * i * a.stride, Run(r < rows ? left : 0, c8 == 0, c8 == 15), tail[i]);
        uint4 bits = make_uint4(0, 0, 0, 0);
        if (RANDOM) bits = philox((uint32_t)row0 + r, (uint32_t)tc * 16 + c8);
        if (TRANSPOSE) {
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4*>(tile + turned<kWords>(r, 4 * c8)) = v[i].r;
            } else {
                *reinterpret_cast<uint4*>(tile + turned<kWords>(r, 8 * c8)) = v[i].r[0];
                *reinterpret_cast<uint4*>(tile + turned<kWords>(r, 8 * c8 + 4)) = v[i].r[1];
            }
            if (RANDOM) *reinterpret_cast<uint4*>(random + turned<kMxTile / 2>(r, 4 * c8)) = bits;
        }
        if (!a.data) continue;
        uint32_t top = largest(v[i]);
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const uint32_t byte = ss::mx_scale<FORMAT>(top);
        // the row's 4 scales of the tile in its first lane
        uint32_t four = byte << (8 * (c8 >> 2));
        four |= __shfl_xor_sync(0xFFFFFFFFu, four, 4);
        four |= __shfl_xor_sync(0xFFFFFFFFu, four, 8);
        if (r < rows) {
            float f[8];
            v[i].get(f);
            const uint32_t words[4] = {bits.x, bits.y, bits.z, bits.w};
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = ss::mx_random<FORMAT>(words[k >> 1], k & 1);
            *reinterpret_cast<Word*>(out) = encode<FORMAT, RANDOM>(f, byte, u);
            if (c8 == 0) *reinterpret_cast<uint32_t*>(scales + 16 * kLines * (i & 3) + 4 * (i >> 2)) = four;
        }
    }
    if (!TRANSPOSE) return;
    __syncthreads();
    // 2 neighbouring threads write a row's 64 elements of the transpose, and their 2 scales
    const int pair = threadIdx.x / kBlocks, block = threadIdx.x % kBlocks;
    const int64_t block0 = part * kBlocks;  // of 32 along the transpose's rows
    Columns<T> c;
    c.load(tile, block, pair);
    uint32_t byte[2];
    c.largest(byte);
#pragma unroll
    for (int j = 0; j < 2; ++j) byte[j] = ss::mx_scale<FORMAT>(byte[j]);
    __align__(16) Word words[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[8] = {};
        if (RANDOM) {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = random[turned<kMxTile / 2>(32 * block + 8 * i + k, pair)];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float f[8];
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[k] = c.get(j, 8 * i + k);
                u[k] = RANDOM ? ss::mx_random<FORMAT>(w[k], j) : 0;
            }
            words[j][i] = encode<FORMAT, RANDOM>(f, byte[j], u);
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t two = byte[j] << (8 * block) | __shfl_xor_sync(0xFFFFFFFFu, byte[j], 1) << (8 * (block ^ 1));
        const int64_t row = col0 + 2 * pair + j;  // of the transpose
        if (row >= a.cols) continue;
        unsigned char* out = a.t_data + row * a.row_tiles * M::kTileRow + (block0 + block) * (M::kTileRow / 4);
#pragma unroll
        for (int i = 0; i < (int)sizeof(words[j]) / 16; ++i)
            reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(words[j])[i];
        if (block == 0)
            *reinterpret_cast<uint16_t*>(a.t_scales + ss::mx_scale_at(row, block0, a.row_tiles)) = (uint16_t)two;
    }
}

struct DequantArgs {
    int64_t rows, cols, col_tiles;
    const unsigned char *data, *scales;
    void* out;
    int64_t stride;
};

template <class T, int FORMAT, int ROUNDS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ DequantArgs a) {
    using M = Mx<FORMAT>;
    using Word = typename M::Word;
    launch_after();
    const int64_t part = blockIdx.x / a.col_tiles, tc = blockIdx.x - part * a.col_tiles;
    const int line = threadIdx.x >> 4, c8 = threadIdx.x & 15;
    const int64_t row0 = part * (kLines * ROUNDS), col = tc * kMxTile + 8 * c8;
    const int rows = (int)min(a.rows - row0, (int64_t)(kLines * ROUNDS)), left = (int)min(a.cols - col, (int64_t)16);
    const int64_t pitch = a.col_tiles * M::kTileRow;
    const unsigned char* data = a.data + (row0 + line) * pitch + tc * M::kTileRow + c8 * (int)sizeof(Word);
    const unsigned char* scales = a.scales + ss::mx_scale_at(row0, 4 * tc + (c8 >> 2), a.col_tiles) + 16 * line;
    wait_before();
    Word w[ROUNDS];
    unsigned char byte[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i, data += kLines * pitch) {
        w[i] = Word();
        byte[i] = 0;
        if (kLines * i + line >= rows || left <= 0) continue;
        w[i] = *reinterpret_cast<const Word*>(data);
        byte[i] = scales[16 * kLines * (i & 3) + 4 * (i >> 2)];
    }
    T* out = static_cast<T*>(a.out) + (row0 + line) * a.stride + col;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i, out += kLines * a.stride) {
        if (kLines * i + (line & ~1) >= rows) break;  // both rows of the warp are behind the last
        float f[8];
        M::decode(w[i], f);
        const float scale = ss::mx_value(byte[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= scale;
        Vec8<T> v;
        v.set(f);
        v.template store<ALIGNED>(out, Run(kLines * i + line < rows ? left : 0, c8 == 0, c8 == 15));
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

// Parts of a matrix by rows where one CTA takes `rounds` loads a thread of them.
int64_t parts(int64_t rows, int rounds) { return (rows + kLines * rounds - 1) / (kLines * rounds); }

// 64 rows a CTA as soon as there are 8 tiles for each SM; below, 16 (fp32 2043 x 1001 to
// 8 bits 5.2 us as tiles, 3.0 as quarters; 1 token of 4096 1.4 us either way).
bool few_tiles(int64_t row_tiles, int64_t col_tiles) { return row_tiles * col_tiles < 8 * (int64_t)ss::num_sms(); }

template <class T, int FORMAT>
int launch_quantize(const QuantArgs& a, bool transpose, bool random, bool aligned, cudaStream_t st) {
    if (!transpose && few_tiles(a.row_tiles, a.col_tiles))
        return with_flags(random, aligned, [&](auto r, auto al) {
            return ss::launch(quantize_kernel<T, FORMAT, kFewRounds, false, decltype(r)::value, decltype(al)::value>,
                              parts(a.rows, kFewRounds) * a.col_tiles, kThreads, 0, 0, true, st, a);
        });
    return with_flags(transpose, random, [&](auto t, auto r) {
        constexpr bool TR = decltype(t)::value, RA = decltype(r)::value;
        constexpr int smem = TR ? tile_bytes<T, RA>() : 0;
        static_assert(smem <= 48 * 1024, "more shared memory has to be asked for");
        const auto kernel = aligned ? quantize_kernel<T, FORMAT, kRounds, TR, RA, true> : quantize_kernel<T, FORMAT, kRounds, TR, RA, false>;
        // the transpose's rows go on to a multiple of 128: parts of whole tiles
        const int64_t by_rows = TR ? a.row_tiles * (kMxTile / kRows) : parts(a.rows, kRounds);
        return ss::launch(kernel, by_rows * a.col_tiles, kThreads, smem, 0, true, st, a);
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
    if (q->stride > INT64_MAX / 8 / q->rows || 8 * tiles(q->rows) * tiles(q->cols) > INT32_MAX) return SS_EOVERFLOW;
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
    if (out_stride > INT64_MAX / 8 / rows || 8 * tiles(rows) * tiles(cols) > INT32_MAX) return SS_EOVERFLOW;
    if (!ss::aligned(out, (uintptr_t)elem_bytes) || !ss::aligned(data, 16) || !ss::aligned(scales, 16)) return SS_EALIGN;
    const DequantArgs a = {rows, cols, tiles(cols), static_cast<const unsigned char*>(data),
                           static_cast<const unsigned char*>(scales), out, out_stride};
    const bool aligned = ss::aligned(out, 16) && out_stride * elem_bytes % 16 == 0;
    return with_flags(format == SS_MXFP4, elem_bytes == 4, [&](auto four, auto wide) {
        constexpr int F = decltype(four)::value ? SS_MXFP4 : SS_MXFP8;
        using T = std::conditional_t<decltype(wide)::value, float, uint16_t>;
        const bool few = few_tiles(tiles(rows), a.col_tiles);
        const auto kernel = few ? (aligned ? dequantize_kernel<T, F, kFewRounds, true> : dequantize_kernel<T, F, kFewRounds, false>)
                                : (aligned ? dequantize_kernel<T, F, kRounds, true> : dequantize_kernel<T, F, kRounds, false>);
        return ss::launch(kernel, parts(rows, few ? kFewRounds : kRounds) * a.col_tiles, kThreads, 0, 0, true,
                          reinterpret_cast<cudaStream_t>(stream), a);
    });
}

}  // extern "C"
