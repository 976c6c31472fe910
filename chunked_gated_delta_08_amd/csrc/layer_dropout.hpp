// layer_dropout.hpp -- which elements dropout keeps: device side of gdn_dropout
// (include/gdn_layer.h), shared by the dropout and the add norm with dropout.
//
// Philox 4x32 with 10 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011), one call for 8 elements of a row, 16 bits
// an element: half the integer work of 32 bits, which beside a pass bound by HBM
// leaves the rate as it is, and steps of 2^-16 in the probability, which the
// factor 1/(1-p) follows exactly.  Where a lane holds four elements (the add norm with an fp32
// residual) two lanes make the same call and take half of its bits each.
#pragma once
#include "layer_launch.hpp"
#include "layer_rows.hpp"

namespace layer {

struct Keep {
    uint32_t key0, key1, off0, off1, drop;   // an element goes where its 16 bits are below `drop`
    float mul;
    __device__ __forceinline__ Keep(const Drop& d) {
        const uint64_t seed = d.rng ? d.rng[0] : d.seed, off = d.rng ? d.rng[1] : d.offset;   // uniform
        key0 = (uint32_t)seed, key1 = (uint32_t)(seed >> 32);
        off0 = (uint32_t)off, off1 = (uint32_t)(off >> 32);
        drop = d.drop, mul = d.mul;
    }
    // The 8 elements of a group: element e's bits are half e % 2 of w[e / 2].
    __device__ __forceinline__ void bits(uint64_t group, uint32_t (&w)[4]) const {
        uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = off0, c3 = off1, k0 = key0, k1 = key1;
#pragma unroll
        for (int i = 0; i < 10; i++) {
            const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
            c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
            c1 = (uint32_t)b;
            c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
            c3 = (uint32_t)a;
            k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
        }
        w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
    }
    __device__ __forceinline__ bool kept(const uint32_t (&w)[4], int e) const {
        return (w[e >> 1] >> 16 * (e & 1) & 0xffff) >= drop;
    }
    // Whether the VEC elements from column c (a multiple of VEC) of a row stay, as bits.
    template <int VEC> __device__ __forceinline__ uint32_t mask(int64_t row, int groups, int c) const {
        static_assert(VEC == 4 || VEC == 8, "a group or half of one");
        uint32_t w[4], m = 0;
        bits((uint64_t)(row * groups + c / 8), w);
        if (VEC == 4 && (c & 4)) w[0] = w[2], w[1] = w[3];
#pragma unroll
        for (int e = 0; e < VEC; e++) m |= (uint32_t)kept(w, e) << e;
        return m;
    }
};

}  // namespace layer
