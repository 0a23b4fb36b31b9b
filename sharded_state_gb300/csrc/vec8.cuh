// vec8.cuh -- 8 consecutive elements of a matrix row, bf16 or fp32, as a thread of the
// row kernels holds them, loaded and stored in 16-byte blocks at any element alignment.
//
// Where rows do not start on 16 bytes, a group's bytes lie in two (bf16) or three
// (fp32) aligned blocks.  Neighbouring lanes hold neighbouring groups of a row, so each
// block is loaded once, by the lane that needs its last bytes, and realigned with the
// next lane's; stores are put together the same way.  (Element by element instead: 1021
// rows of 1001 bf16, forward and backward 58 us where this takes less than half.)
#pragma once

#include <cstdint>

#include "device_utils.cuh"
#include "segmap.cuh"

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

__device__ __forceinline__ uint4 from_next_lane(uint4 v) {
    return make_uint4(__shfl_down_sync(0xFFFFFFFFu, v.x, 1), __shfl_down_sync(0xFFFFFFFFu, v.y, 1),
                      __shfl_down_sync(0xFFFFFFFFu, v.z, 1), __shfl_down_sync(0xFFFFFFFFu, v.w, 1));
}

// Words [lo, hi) of the 16-byte value v to blk.
__device__ __forceinline__ void st_words(unsigned char* blk, uint4 v, int lo, int hi) {
    uint32_t* w = reinterpret_cast<uint32_t*>(blk);
    if (lo <= 0 && hi > 0) w[0] = v.x;
    if (lo <= 1 && hi > 1) w[1] = v.y;
    if (lo <= 2 && hi > 2) w[2] = v.z;
    if (lo <= 3 && hi > 3) w[3] = v.w;
}

// The first `bytes` (even, up to 14) of an aligned 16-byte block, or its last ones.
__device__ __forceinline__ void st_head(unsigned char* blk, uint4 v, int bytes) {
    if (bytes & 8) *reinterpret_cast<uint2*>(blk) = make_uint2(v.x, v.y);
    const uint32_t w = bytes & 8 ? v.z : v.x, x = bytes & 8 ? v.w : v.y;
    blk += bytes & 8;
    if (bytes & 4) *reinterpret_cast<uint32_t*>(blk) = w;
    if (bytes & 2) *reinterpret_cast<uint16_t*>(blk + (bytes & 4)) = (uint16_t)(bytes & 4 ? x : w);
}
__device__ __forceinline__ void st_tail(unsigned char* blk, uint4 v, int bytes) {
    if (bytes & 8) *reinterpret_cast<uint2*>(blk + 8) = make_uint2(v.z, v.w);
    const uint32_t w = bytes & 8 ? v.y : v.w, x = bytes & 8 ? v.x : v.z;
    blk += bytes & 8 ? 8 : 16;
    if (bytes & 4) *reinterpret_cast<uint32_t*>(blk - 4) = w;
    if (bytes & 2) *reinterpret_cast<uint16_t*>(blk - (bytes & 4) - 2) = (uint16_t)((bytes & 4 ? x : w) >> 16);
}

// A lane's place in its row: n elements of its own (0: none), `after` in the next lane
// (0 where that is not the group behind this one), and whether the lane before holds
// the group before.
struct Run {
    int n, after;
    bool prev;

    // left: elements of the row from this group on (any sign); first, last: of the
    // lanes that hold neighbouring groups.
    __device__ __forceinline__ Run(int left, bool first, bool last)
        : n(max(0, min(left, 8))), after(last ? 0 : max(0, min(left - 8, 8))), prev(!first && left > 0) {}
};

template <class T>
struct Vec8;

// Loads and stores with ALIGNED want p on 16 bytes; without, the whole warp makes them.
// A load is in two steps, so that many can be on their way: fetch() asks for the blocks
// (`tail` for one that no other lane loads), settle() of the same p and run makes of them
// the lane's n elements, zeros behind them.
template <>
struct Vec8<uint16_t> {  // bf16
    uint4 r;

    __device__ __forceinline__ void clear() { r = make_uint4(0, 0, 0, 0); }

    template <bool ALIGNED>
    __device__ __forceinline__ void fetch(const uint16_t* p, const Run& run, uint4& tail) {
        const int sh = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        const unsigned char* blk = reinterpret_cast<const unsigned char*>(p) - sh;
        r = make_uint4(0, 0, 0, 0);
        if (run.n > 0) r = ld_row_u4(blk);
        if (!ALIGNED && run.after == 0 && sh + 2 * run.n > 16) tail = ld_row_u4(blk + 16);
    }

    template <bool ALIGNED>
    __device__ __forceinline__ void settle(const uint16_t* p, const Run& run, const uint4& tail) {
        if (!ALIGNED) {
            const uint4 next = from_next_lane(r);
            r = realign16(r, run.after == 0 ? tail : next, (int)(reinterpret_cast<uintptr_t>(p) & 15u));
        }
        if (run.n < 8) {
            r.x = run.n > 1 ? r.x : run.n > 0 ? r.x & 0xFFFFu : 0u;
            r.y = run.n > 3 ? r.y : run.n > 2 ? r.y & 0xFFFFu : 0u;
            r.z = run.n > 5 ? r.z : run.n > 4 ? r.z & 0xFFFFu : 0u;
            r.w = run.n > 6 ? r.w & 0xFFFFu : 0u;
        }
    }

    template <bool ALIGNED>
    __device__ __forceinline__ void load(const uint16_t* p, const Run& run) {
        uint4 tail = make_uint4(0, 0, 0, 0);
        fetch<ALIGNED>(p, run, tail);
        settle<ALIGNED>(p, run, tail);
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
    __device__ __forceinline__ void store(uint16_t* p, const Run& run) const {
        unsigned char* c = reinterpret_cast<unsigned char*>(p);
        const int sh = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        uint4 next = make_uint4(0, 0, 0, 0);
        if (!ALIGNED) next = from_next_lane(r);
        if (run.n == 0) return;
        if (sh == 0) {
            if (run.n == 8)
                *reinterpret_cast<uint4*>(p) = r;
            else
                st_head(c, r, 2 * run.n);
            return;
        }
        const int head = 16 - sh;  // bytes that go into the block before
        if (run.n == 8 && 2 * run.after >= head)
            *reinterpret_cast<uint4*>(c + head) = realign16(r, next, head);
        else if (2 * run.n > head)
            st_head(c + head, realign16(r, r, head), 2 * run.n - head);
        if (run.prev && 2 * run.n >= head) return;  // the lane before has written them
        if (2 * run.n >= head)
            st_tail(c - sh, realign16(r, r, head), head);
        else  // both ends inside one block
            st_bytes(c - sh, realign16(r, r, head), sh, sh + 2 * run.n);
    }
};

template <>
struct Vec8<float> {
    uint4 r[2];

    __device__ __forceinline__ void clear() { r[0] = r[1] = make_uint4(0, 0, 0, 0); }

    template <bool ALIGNED>
    __device__ __forceinline__ void fetch(const float* p, const Run& run, uint4& tail) {
        const int sh = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        const unsigned char* blk = reinterpret_cast<const unsigned char*>(p) - sh;
        clear();
        if (run.n > 0) r[0] = ld_row_u4(blk);
        if (sh + 4 * run.n > 16) r[1] = ld_row_u4(blk + 16);
        if (!ALIGNED && run.after == 0 && sh + 4 * run.n > 32) tail = ld_row_u4(blk + 32);
    }

    template <bool ALIGNED>
    __device__ __forceinline__ void settle(const float* p, const Run& run, const uint4& tail) {
        if (!ALIGNED) {
            const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
            const uint4 next = from_next_lane(r[0]);
            r[0] = realign16(r[0], r[1], sh);
            r[1] = realign16(r[1], run.after == 0 ? tail : next, sh);
        }
        if (run.n < 8) {
            r[0].x = run.n > 0 ? r[0].x : 0u, r[0].y = run.n > 1 ? r[0].y : 0u;
            r[0].z = run.n > 2 ? r[0].z : 0u, r[0].w = run.n > 3 ? r[0].w : 0u;
            r[1].x = run.n > 4 ? r[1].x : 0u, r[1].y = run.n > 5 ? r[1].y : 0u;
            r[1].z = run.n > 6 ? r[1].z : 0u, r[1].w = 0u;
        }
    }

    template <bool ALIGNED>
    __device__ __forceinline__ void load(const float* p, const Run& run) {
        uint4 tail = make_uint4(0, 0, 0, 0);
        fetch<ALIGNED>(p, run, tail);
        settle<ALIGNED>(p, run, tail);
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
    __device__ __forceinline__ void store(float* p, const Run& run) const {
        unsigned char* c = reinterpret_cast<unsigned char*>(p);
        const int sh = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        uint4 next = make_uint4(0, 0, 0, 0);
        if (!ALIGNED) next = from_next_lane(r[0]);
        if (run.n == 0) return;
        if (sh == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (run.n >= 4 * i + 4)
                    *reinterpret_cast<uint4*>(c + 16 * i) = r[i];
                else
                    st_words(c + 16 * i, r[i], 0, run.n - 4 * i);
            }
            return;
        }
        const int head = 16 - sh, words = head >> 2;  // that go into the block before
        const uint4 first = realign16(r[0], r[1], head), second = realign16(r[1], next, head);
        if (run.n >= words + 4)
            *reinterpret_cast<uint4*>(c + head) = first;
        else
            st_words(c + head, first, 0, run.n - words);
        if (run.n == 8 && run.after >= words)
            *reinterpret_cast<uint4*>(c + head + 16) = second;
        else
            st_words(c + head + 16, second, 0, run.n - words - 4);
        if (!run.prev || run.n < words) st_words(c - sh, realign16(r[0], r[0], head), sh >> 2, min(4, (sh >> 2) + run.n));
    }
};

}  // namespace ss
