// philox.cuh -- the counter-based generator behind dropout and stochastic
// rounding: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011).
//
// The key is the caller's seed, the counter {column / 8, row, offset}: an
// element's bits follow from its place in the matrix and from nothing else, so
// nothing of a mask is stored and a backward pass, or a kernel that takes other
// elements at a time, makes the same ones again.  Each call's 128 bits serve the
// 8 elements that a thread loads at once, 16 bits each: a probability in steps of
// 2^-16, and half the generator's arithmetic of 32 bits each.
#pragma once

#include <cstdint>

namespace ss {

struct Philox {
    uint32_t key0, key1, off0, off1;

    Philox() = default;

    // rng: {seed, offset} on the device.  Every lane keeps them as values of its own: put
    // through a warp reduction first (one value for all lanes, in uniform registers), wrong
    // masks came out of the norm's unaligned forward instances that spill registers, of no
    // other, and it was no faster.
    __device__ __forceinline__ explicit Philox(const int64_t* rng) {
        const uint64_t seed = (uint64_t)rng[0], offset = (uint64_t)rng[1];
        key0 = (uint32_t)seed, key1 = (uint32_t)(seed >> 32);
        off0 = (uint32_t)offset, off1 = (uint32_t)(offset >> 32);
    }

    // The 128 bits of columns 8 group .. 8 group + 7 of a row, lowest first.
    __device__ __forceinline__ uint4 operator()(uint32_t row, uint32_t group) const {
        uint32_t a = group, b = row, c = off0, d = off1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p = (uint64_t)0xD2511F53u * a, q = (uint64_t)0xCD9E8D57u * c;
            a = (uint32_t)(q >> 32) ^ b ^ (key0 + i * 0x9E3779B9u);
            c = (uint32_t)(p >> 32) ^ d ^ (key1 + i * 0xBB67AE85u);
            b = (uint32_t)q;
            d = (uint32_t)p;
        }
        return make_uint4(a, b, c, d);
    }
};

// 8 floats with their dropout: kept, and scaled, where their 16 bits are `drop` or
// more.  A dropped element is 0 whatever it held.
__device__ __forceinline__ void drop8(float (&x)[8], uint4 bits, uint32_t drop, float scale) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w}, least = drop << 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = (w[i] << 16) >= least ? __fmul_rn(x[2 * i], scale) : 0.f;
        x[2 * i + 1] = w[i] >= least ? __fmul_rn(x[2 * i + 1], scale) : 0.f;
    }
}

}  // namespace ss
