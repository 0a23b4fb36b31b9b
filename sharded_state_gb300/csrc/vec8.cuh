// vec8.cuh -- 8 consecutive elements of a matrix row, bf16 or fp32, at any element
// alignment, as a thread of the row kernels holds them.
#pragma once

#include <cstdint>

#include "device_utils.cuh"

namespace ss {

// Loads that may be of data the same kernel overwrites (in-place calls): not .nc.
__device__ __forceinline__ uint4 ld_row_u4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

template <class T>
struct Vec8;

template <>
struct Vec8<uint16_t> {  // bf16
    uint4 r;

    __device__ __forceinline__ void clear() { r = make_uint4(0, 0, 0, 0); }

    // Elements [0, n) of the 8 at p, the others 0.  ALIGNED: p is on 16 bytes.
    template <bool ALIGNED>
    __device__ __forceinline__ void load(const uint16_t* p, int n) {
        if (ALIGNED && n >= 8) {
            r = ld_row_u4(p);
            return;
        }
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 1] |= (uint32_t)*reinterpret_cast<const volatile uint16_t*>(p + i) << (16 * (i & 1));
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }

    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = bf16_lo(r.x), f[1] = bf16_hi(r.x), f[2] = bf16_lo(r.y), f[3] = bf16_hi(r.y);
        f[4] = bf16_lo(r.z), f[5] = bf16_hi(r.z), f[6] = bf16_lo(r.w), f[7] = bf16_hi(r.w);
    }

    // Rounded to the nearest, ties to even.
    __device__ __forceinline__ void set(const float (&f)[8]) {
        r = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }

    template <bool ALIGNED>
    __device__ __forceinline__ void store(uint16_t* p, int n) const {
        if (ALIGNED && n >= 8) {
            *reinterpret_cast<uint4*>(p) = r;
            return;
        }
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
};

template <>
struct Vec8<float> {
    uint4 r[2];

    __device__ __forceinline__ void clear() { r[0] = r[1] = make_uint4(0, 0, 0, 0); }

    template <bool ALIGNED>
    __device__ __forceinline__ void load(const float* p, int n) {
        if (ALIGNED && n >= 8) {
            r[0] = ld_row_u4(p);
            r[1] = ld_row_u4(p + 4);
            return;
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = i < n ? *reinterpret_cast<const volatile uint32_t*>(p + i) : 0u;
        r[0] = make_uint4(w[0], w[1], w[2], w[3]);
        r[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }

    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(r[i].x), f[4 * i + 1] = __uint_as_float(r[i].y);
            f[4 * i + 2] = __uint_as_float(r[i].z), f[4 * i + 3] = __uint_as_float(r[i].w);
        }
    }

    __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                              __float_as_uint(f[4 * i + 3]));
    }

    template <bool ALIGNED>
    __device__ __forceinline__ void store(float* p, int n) const {
        if (ALIGNED && n >= 8) {
            *reinterpret_cast<uint4*>(p) = r[0];
            *reinterpret_cast<uint4*>(p + 4) = r[1];
            return;
        }
        const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = __uint_as_float(w[i]);
    }
};

}  // namespace ss
