// mx.cuh -- microscaled floats as the OCP Microscaling Formats specification (v1.0)
// defines them: 32 consecutive elements of a row share a power of two, e2m1 elements
// (MXFP4) or e4m3 elements (MXFP8) hold the rest.
//
// A block's scale is 2^(floor(log2 max|x|) - e), e the exponent of the format's
// largest element (2 or 8), stored as its exponent + 127; elements beyond the largest
// saturate.  Scaling by a power of two is exact, so a quantised element is one
// rounding away from its input.  A block with an infinity or a NaN in it has the
// scale NaN (255) and stands for NaN throughout: it is never quietly finite.
//
// Layout (what the tensor cores read as it is):
//   data    rows of whole 128 elements, the ones past the end zero: 64 or 128 bytes
//           for each 128; of two e2m1 elements in a byte the first is the low half
//   scales  512 bytes for each 128 rows x 128 columns, tiles of a row of tiles one
//           after the other: the 4 scales of row r at 16 (r % 32) + 4 (r / 32)
#pragma once

#include <cstdint>

#include "shardstate.h"

namespace ss {

constexpr int kMxBlock = 32;   // elements of a scale
constexpr int kMxTile = 128;   // rows and columns of a tile of scales
constexpr int kMxTileBytes = 512;

template <int FORMAT>
struct Mx;

template <>
struct Mx<SS_MXFP4> {
    static constexpr int kTop = 2;        // exponent of the largest element
    static constexpr int kLowest = 0;     // lowest exponent of a normal element
    static constexpr int kFraction = 1;   // bits
    static constexpr int kBits = 4;
    static constexpr int kTileRow = 64;   // bytes of 128 elements
    using Word = uint32_t;                // 8 elements

    // 8 elements, rounded to the nearest (ties to even) and saturated.
    __device__ static __forceinline__ Word encode(const float (&f)[8]) {
        uint32_t w;
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(w)
            : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
        return w;
    }

    __device__ static __forceinline__ void decode(Word w, float (&f)[8]) {
        uint32_t h[4];
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(w));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
                : "r"(h[i]));
    }
};

template <>
struct Mx<SS_MXFP8> {
    static constexpr int kTop = 8;
    static constexpr int kLowest = -6;
    static constexpr int kFraction = 3;
    static constexpr int kBits = 8;
    static constexpr int kTileRow = 128;
    using Word = uint2;

    __device__ static __forceinline__ Word encode(const float (&f)[8]) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 a, b;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
                "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
                "mov.b32 %0, {a, b};\n\t}"
                : "=r"(w[i])
                : "f"(f[4 * i]), "f"(f[4 * i + 1]), "f"(f[4 * i + 2]), "f"(f[4 * i + 3]));
        return make_uint2(w[0], w[1]);
    }

    __device__ static __forceinline__ void decode(Word v, float (&f)[8]) {
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 a, b, c, d;\n\t.reg .b32 x, y;\n\t"
                "mov.b32 {a, b}, %4;\n\t"
                "cvt.rn.f16x2.e4m3x2 x, a;\n\t"
                "cvt.rn.f16x2.e4m3x2 y, b;\n\t"
                "mov.b32 {a, b}, x;\n\tmov.b32 {c, d}, y;\n\t"
                "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\tcvt.f32.f16 %2, c;\n\tcvt.f32.f16 %3, d;\n\t}"
                : "=f"(f[4 * i]), "=f"(f[4 * i + 1]), "=f"(f[4 * i + 2]), "=f"(f[4 * i + 3])
                : "r"(w[i]));
    }
};

// |x| as its bits, which order like the magnitudes do, NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The stored scale of a block whose largest magnitude has these bits.  (A subnormal
// maximum is below 2^-126 and the lowest scale, 2^-127, is the one to take.)
template <int FORMAT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t largest) {
    const int e = (int)(largest >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - Mx<FORMAT>::kTop, 0);
}

// 1 / scale (of one that is not NaN).
__device__ __forceinline__ float mx_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// The scale's value.
__device__ __forceinline__ float mx_value(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FFFFFFFu)
                        : byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Byte of the scale of row r, block b (of 32 columns) in a matrix `tiles` tiles wide.
__device__ __forceinline__ int64_t mx_scale_at(int64_t r, int64_t b, int64_t tiles) {
    return ((r >> 7) * tiles + (b >> 2)) * kMxTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// The lower or upper 16 random bits of a word as mx_encode_random takes them: in the
// middle bytes, behind a code in the top one, with what the codes begin with in fp32
// taken off there (252 or 192 of 256, so 4 or 64 to be added).
template <int FORMAT>
__device__ __forceinline__ uint32_t mx_random(uint32_t word, bool upper) {
    return __byte_perm(word, Mx<FORMAT>::kBits == 4 ? 0x04000000u : 0x40000000u, upper ? 0x7324 : 0x7104);
}

// 8 elements times `inverse`, rounded down or up in magnitude: up where what is cut off
// and the element's 16 random bits / 2^16 make one step.  In the format's normal range
// the codes are the leading bits of the fp32 magnitude, and the random bits, added right
// behind them, carry into them just then; below it the lowest normal number is added
// first, which puts every element on the same steps, and half of the sum, which is more
// than the element there and no more above, has the leading bits that continue the codes
// (towards zero, so that nothing is rounded but by the cut).  The sums' top bytes are the
// codes; one past the largest is put right for all of them at once.
template <int FORMAT>
__device__ __forceinline__ typename Mx<FORMAT>::Word mx_encode_random(const float (&f)[8], float inverse,
                                                                      const uint32_t (&random)[8]) {
    using M = Mx<FORMAT>;
    constexpr int kCut = 23 - M::kFraction;
    static_assert(((127 + M::kLowest - 1) << M::kFraction) % 256 == (M::kBits == 4 ? 252 : 192), "mx_random");
    const float least = __uint_as_float((uint32_t)(127 + M::kLowest) << 23);
    uint32_t sum[8], sign[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = fabsf(f[i]) * inverse;
        const float t = fmaxf(v, __fmaf_rz(v, 0.5f, 0.5f * least));
        sum[i] = __float_as_uint(t) * (1u << (24 - kCut)) + random[i];
        sign[i] = __float_as_uint(f[i]);
    }
    // top bytes, four at a time
    auto top = [](const uint32_t (&x)[8], int i, int step) {
        return __byte_perm(__byte_perm(x[i], x[i + step], 0x0073), __byte_perm(x[i + 2 * step], x[i + 3 * step], 0x0073),
                           0x5410);
    };
    typename M::Word out;
    if constexpr (M::kBits == 4) {
        const uint32_t w = top(sum, 0, 2) + top(sum, 1, 2) * 16u;
        out = (w - (w >> 3 & 0x11111111u)) | (top(sign, 0, 2) >> 4 & 0x08080808u) | (top(sign, 1, 2) & 0x80808080u);  // 8 -> 7
    } else {
        uint32_t w[2] = {top(sum, 0, 1), top(sum, 4, 1)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // 0x7F, 0x80 -> 0x7E
            const uint32_t over = (((w[i] + 0x01010101u) | w[i]) & 0x80808080u) >> 7;
            w[i] = (w[i] & ~(over * 0xFFu)) | over * 0x7Eu;
        }
        out = make_uint2(w[0] | (top(sign, 0, 1) & 0x80808080u), w[1] | (top(sign, 4, 1) & 0x80808080u));
    }
    return out;
}

// 8 elements times `inverse`, to the nearest.
template <int FORMAT>
__device__ __forceinline__ typename Mx<FORMAT>::Word mx_encode(const float (&f)[8], float inverse) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = f[i] * inverse;
    return Mx<FORMAT>::encode(g);
}

}  // namespace ss
