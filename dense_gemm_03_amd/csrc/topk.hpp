// The largest values of a stream, kept by one wave: a list of 64 keys in falling
// order, one per lane.
//
// A key is 64 bits, the value's order above, the complement of its place below:
// keys are distinct, and equal values rank by the lower place.  0 is no key.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

// Bits of v in the order of the numbers; -0 as +0, NaN as -infinity.
__device__ __forceinline__ uint32_t order_of(float v)
{
    const float z = v != v ? -__builtin_inff() : v + 0.0f;
    const uint32_t b = __float_as_uint(z);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order)
{
    return __uint_as_float(order ^ ((uint32_t)((int32_t)~order >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t key_of(float v, int place)
{
    return (uint64_t)order_of(v) << 32 | (uint32_t)~place;
}
__device__ __forceinline__ int place_of(uint64_t key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ uint64_t key_xor_lane(uint64_t v, int mask)
{
    return (uint64_t)(uint32_t)__shfl_xor((int)(v >> 32), mask) << 32 | (uint32_t)__shfl_xor((int)v, mask);
}
__device__ __forceinline__ uint64_t key_at(uint64_t v, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
// The key of the lane below (lane 0: its own).
__device__ __forceinline__ uint64_t key_from_below(uint64_t v)
{
    const int hi = (int)(v >> 32), lo = (int)v;
    return (uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(hi, hi, 0x138, 0xf, 0xf, false) << 32 |
           (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, 0x138, 0xf, 0xf, false);
}

__device__ __forceinline__ uint64_t exchange(uint64_t v, int lane, int j, bool falling)
{
    const uint64_t o = key_xor_lane(v, j);
    const bool larger = ((lane & j) == 0) == falling;   // which of the two this lane keeps
    return (v > o) == larger ? v : o;
}

// 64 keys, one per lane, in falling order (bitonic: 21 exchanges).
__device__ __forceinline__ uint64_t sorted(uint64_t v, int lane)
{
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) v = exchange(v, lane, j, (lane & k) == 0);
    return v;
}

// The 64 largest of two falling lists, falling: the first against the second
// turned round gives them in bitonic order, 6 exchanges sort it.
__device__ __forceinline__ uint64_t merged(uint64_t a, uint64_t b, int lane)
{
    const uint64_t r = key_xor_lane(b, 63);
    uint64_t v = a > r ? a : r;
#pragma unroll
    for (int j = 32; j > 0; j >>= 1) v = exchange(v, lane, j, true);
    return v;
}

struct TopList {
    uint64_t list = 0;     // lane i: the i-th largest so far
    uint64_t least = 0;    // the top-th of them: what a key has to exceed
    int lane, top;

    __device__ __forceinline__ TopList(int lane_, int top_) : lane(lane_), top(top_) {}

    __device__ __forceinline__ void merge(uint64_t falling)
    {
        list = merged(list, falling, lane);
        least = key_at(list, top - 1);
    }
    __device__ __forceinline__ void insert(uint64_t key)   // the same key in all lanes
    {
        const int at = __builtin_popcountll(__ballot(list > key));
        const uint64_t below = key_from_below(list);
        list = lane < at ? list : lane == at ? key : below;
        least = key_at(list, top - 1);
    }
    // N keys per lane, key(j) for j < N (0: none).  If many lanes have one for the
    // list, the lanes' largest go in at once, sorted; that leaves few others above
    // the new bound, and those are put in one by one.
    template <int N, class Key>
    __device__ __forceinline__ void absorb(Key &&key)
    {
        uint64_t best = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t k = key(j);
            best = k > best ? k : best;
        }
        const int lanes = __builtin_popcountll(__ballot(best > least));
        if (lanes == 0) return;
        if (lanes > 6)
            merge(sorted(best > least ? best : 0, lane));
        else
            best = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t k = key(j);
            uint64_t rest = __ballot(k > least && k != best);
            while (rest != 0) {
                const int at = __builtin_ctzll(rest);
                insert(key_at(k, at));
                rest &= __ballot(k > least) & ~(1ull << at);
            }
        }
    }
};

}  // namespace dg
