// The largest values of a stream, kept by one wave: a list of 64 keys in falling
// order, one per lane.
//
// A key is 64 bits, the value's order above, the complement of its place below:
// keys are distinct, and equal values rank by the lower place.  0 is no key.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "strip.hpp"

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

// v of the lane whose number differs in the bits `mask`, through the vector unit:
// DPP within 16 lanes, swaps of rows and halves beyond.  (Through LDS, as a shuffle, a
// sort took twice as long: 131072 logits with 20 alternatives 16.5 us, then 14.)
template <int MASK>
__device__ __forceinline__ uint32_t xor_lane(uint32_t v)
{
    if constexpr (MASK == 1) return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xf, 0xf, false);        // quad_perm 1 0 3 2
    if constexpr (MASK == 2) return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xf, 0xf, false);        // quad_perm 2 3 0 1
    if constexpr (MASK == 3) return __builtin_amdgcn_update_dpp(v, v, 0x1B, 0xf, 0xf, false);        // quad_perm 3 2 1 0
    if constexpr (MASK == 7) return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xf, 0xf, false);       // row_half_mirror
    if constexpr (MASK == 8) return __builtin_amdgcn_update_dpp(v, v, 0x128, 0xf, 0xf, false);       // row_ror:8
    if constexpr (MASK == 15) return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xf, 0xf, false);      // row_mirror
    if constexpr (MASK == 4) return xor_lane<3>(xor_lane<7>(v));
    if constexpr (MASK == 16 || MASK == 32) {
        // both operands v: the odd rows (the upper half) of the first and the even
        // rows (the lower half) of the second change places
        const auto r = MASK == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                                  : __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)) & MASK ? r[0] : r[1];
    }
    if constexpr (MASK == 63) return xor_lane<32>(xor_lane<16>(xor_lane<15>(v)));
}
template <int MASK>
__device__ __forceinline__ uint64_t key_xor_lane(uint64_t v)
{
    return (uint64_t)xor_lane<MASK>((uint32_t)(v >> 32)) << 32 | xor_lane<MASK>((uint32_t)v);
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

// The lanes that keep the smaller key when lanes that differ in bit J compare, in
// blocks of K lanes that fall and rise in turn (K == 64: all fall).
__host__ __device__ constexpr uint64_t keeps_smaller(int j, int k)
{
    uint64_t m = 0;
    for (int lane = 0; lane < 64; ++lane)
        if (((lane & j) == 0) != ((lane & k) == 0)) m |= 1ull << lane;
    return m;
}

// The steps of a bitonic sort over lanes that differ in bit J and below.
template <int J, int K>
__device__ __forceinline__ uint64_t exchanged(uint64_t v)
{
    const uint64_t o = key_xor_lane<J>(v);
    // a constant mask: formed from the lane's number, the masks of all steps took
    // 56 registers, and spilled
    constexpr uint64_t SMALLER = keeps_smaller(J, K);
    v = __builtin_amdgcn_inverse_ballot_w64(__ballot(v > o) ^ SMALLER) ? v : o;
    if constexpr (J > 1) v = exchanged<J / 2, K>(v);
    return v;
}

// 64 keys, one per lane, in falling order (bitonic: 21 exchanges).
__device__ __forceinline__ uint64_t sorted(uint64_t v)
{
    return exchanged<32, 64>(
        exchanged<16, 32>(exchanged<8, 16>(exchanged<4, 8>(exchanged<2, 4>(exchanged<1, 2>(v))))));
}

// The 64 largest of two falling lists, falling: the first against the second
// turned round gives them in bitonic order, 6 exchanges sort it.
__device__ __forceinline__ uint64_t merged(uint64_t a, uint64_t b)
{
    const uint64_t r = key_xor_lane<63>(b);
    return exchanged<32, 64>(a > r ? a : r);
}

struct TopList {
    uint64_t list = 0;     // lane i: the i-th largest so far
    uint64_t least = 0;    // the top-th of them: what a key has to exceed
    int lane, top;

    __device__ __forceinline__ TopList(int lane_, int top_) : lane(lane_), top(top_) {}

    __device__ __forceinline__ void merge(uint64_t falling)
    {
        list = merged(list, falling);
        least = key_at(list, top - 1);
    }
    __device__ __forceinline__ void insert(uint64_t key)   // the same key in all lanes
    {
        const int at = __builtin_popcountll(__ballot(list > key));
        const uint64_t below = key_from_below(list);
        list = lane < at ? list : lane == at ? key : below;
        least = key_at(list, top - 1);
    }
    // N values per lane, v[j] at place(first, j) (not below 0 and below n, or the value
    // does not count and is -infinity), `largest` the lane's largest, as fmaxf finds it.
    // If many lanes have something for the list, their largest go in at once, sorted,
    // which leaves little above the new bound.  The lanes that have something (else),
    // mostly one or two, are gone through one by one, their N values spread over the
    // lanes through `row` (LDS, N floats of this wave's own).
    template <int N, class Place>
    __device__ __forceinline__ void absorb_values(const float (&v)[N], float largest, int n, int first, Place &&place,
                                                  float *row)
    {
        static_assert(N <= 64 && N % 4 == 0, "a lane's values fit the wave");
        uint64_t best = 0;            // this lane's key that is in the list already
        uint64_t lanes = __ballot(least == 0 || largest > value_of((uint32_t)(least >> 32)));
        if (least == 0 || __builtin_popcountll(lanes) > MANY) {
            // the largest value's first place; NaN and -infinity, which fmaxf does not tell apart, are left to the rest
            const float none = -__builtin_inff();
            int at = 0;
#pragma unroll
            for (int j = N - 1; j >= 0; --j) at = v[j] == largest ? place(first, j) : at;
            best = largest > none ? key_of(largest, at) : 0;
            merge(sorted(best > least ? best : 0));
            const float bar = value_of((uint32_t)(least >> 32));
            int count = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) count += v[j] >= bar;
            lanes = least == 0 || bar == none ? ~0ull : __ballot(count > (best != 0 ? 1 : 0));
        }
        while (lanes != 0) {
            const int from = __builtin_ctzll(lanes);
            lanes &= lanes - 1;
            if (lane == from) {
#pragma unroll
                for (int j = 0; j < N; ++j) row[j] = v[j];
            }
            wave_order();
            const int at = place(__builtin_amdgcn_readlane(first, from), lane % N);
            const float value = row[lane % N];
            wave_order();
            const uint64_t k = lane < N && (unsigned)at < (unsigned)n ? key_of(value, at) : 0;
            insert_lanes(k != key_at(best, from) ? k : 0);
        }
    }

private:
    // Lanes from which a sort costs less than insertions: 27 exchanges against one
    // insertion per value.
    static constexpr int MANY = 6;

    // each lane's key, one by one
    __device__ __forceinline__ void insert_lanes(uint64_t k)
    {
        uint64_t rest = __ballot(k > least);
        while (rest != 0) {
            const int at = __builtin_ctzll(rest);
            insert(key_at(k, at));
            rest &= __ballot(k > least) & ~(1ull << at);
        }
    }
};

}  // namespace dg
