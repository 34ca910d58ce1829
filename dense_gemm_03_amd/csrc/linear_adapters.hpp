// Low-rank adapters in the linear layers' kernels: after a block's product its sums
// take up t . b^T, with t = scale x . a^T of the row's own adapter (adapter.hip forms
// it before the product).
//
// The ranks are a few k-steps more, so they cost the product little as MFMAs, but a
// tile may hold rows of several adapters: it goes through the adapters of its rows, each
// with the rows of t that are not its own as zeros.  Rows of a request lie together, so
// that is one or two adapters for most tiles; where every row has another one, what
// counts is how many of their b are on the way at a time.
//
// Measured, with the first product: 4096 rows of 8 requests, 4096 x 8192, rank 64: 258 us,
// 211 without adapters; 1 row, 4096 x 4096, rank 16: 14 us and 7.6.
//
// bf16 products read t as a sum of two bf16 values (16 bits of it: two MFMAs instead
// of one, on the few steps that the ranks take).
#pragma once

#include "mma16.hpp"

namespace dg {

struct AdapterArgs {
    const void *t;          // rows x pitch; bf16: the upper halves, and `plane` elements on the lower ones
    const void *b;          // per adapter N x rank
    const int32_t *ids;     // per row; outside 0 .. count-1: none
    int64_t ldb, stride_b;
    int64_t plane;
    int count, rank, pitch; // pitch: whole 16 bytes
    // parts > 0: t is not formed yet, but the fp32 sums of parts of K, `plane` elements apart
    // (a few rows, for which a launch costs more than adding them up where they are used;
    // kernels of tiles larger than 64 x 64 have no registers for that)
    int parts;
};

constexpr int ADAPTER_MAX_PARTS = 8;

// KV values of k from e0 of a row, zero from `end` on.
template <bool BF16>
struct AdapterOperand {
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    static constexpr int KV = BF16 ? 8 : 4, PLANES = BF16 ? 2 : 1;
    typedef In chunk __attribute__((ext_vector_type(KV), aligned(sizeof(In))));

    static constexpr uint32_t LARGE = BF16 ? 0x7F007F00u : 0x7F000000u;      // 2^127: its square is infinite
    static constexpr uint32_t EXPONENT = BF16 ? 0x7F807F80u : 0x7F800000u;   // all ones: infinity or NaN

    // The largest exponents of `so_far` and v (bf16: of each half).
    static __device__ __forceinline__ uint32_t largest(uint32_t so_far, const u32x4 &v)
    {
        typedef uint16_t pair __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t e = v[d] & EXPONENT;
            so_far = BF16 ? __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(pair, so_far),
                                                                                   __builtin_bit_cast(pair, e)))
                          : max(so_far, e);
        }
        return so_far;
    }
    static __device__ __forceinline__ bool infinite(uint32_t exponents)
    {
        return BF16 ? exponents >> 16 == 0x7F80u || (exponents & 0xFFFFu) == 0x7F80u : exponents == EXPONENT;
    }
    static __device__ __forceinline__ uint32_t not_finite(uint32_t v)   // all ones in the places of such values
    {
        if (!BF16) return infinite(v & EXPONENT) ? ~0u : 0u;
        return (infinite(v & 0x7F80u) ? 0xFFFFu : 0u) | (infinite(v & 0x7F800000u) ? 0xFFFF0000u : 0u);
    }
    // v with zeros for values that are not finite; or their marks: LARGE in their places, else 0.
    static __device__ __forceinline__ u32x4 apart(u32x4 v, bool marks)
    {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t out = not_finite(v[d]);
            v[d] = marks ? LARGE & out : v[d] & ~out;
        }
        return v;
    }
    template <class Sum>
    static __device__ __forceinline__ void mma(const u32x4 &a, const u32x4 &v, Sum &sum)
    {
        if constexpr (BF16) {
            sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, v), sum,
                                                          0, 0, 0);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                sum = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[d]), __uint_as_float(v[d]), sum, 0, 0, 0);
        }
    }
    // b, at the element's alignment
    static __device__ __forceinline__ u32x4 load(const In *row, int e0, int end)
    {
        if (e0 + KV <= end) return __builtin_bit_cast(u32x4, *reinterpret_cast<const chunk *>(row + e0));
        if (e0 >= end) return u32x4{0, 0, 0, 0};
        union {
            u32x4 v;
            In e[KV];
        } u;
#pragma unroll
        for (int i = 0; i < KV; ++i) u.e[i] = e0 + i < end ? row[e0 + i] : In(0);
        return u.v;
    }
    // The same from parts.
    static __device__ __forceinline__ void load_parts(const AdapterArgs &p, bool has, int64_t row, int e0, u32x4 (&v)[PLANES])
    {
        const float *t = static_cast<const float *>(p.t) + row * p.pitch + e0;
        float sum[KV];
#pragma unroll
        for (int i = 0; i < KV; ++i) sum[i] = 0.0f;
        if (has && e0 < p.rank) {
            // all on the way together; behind the last part, that one again
            u32x4 w[ADAPTER_MAX_PARTS][KV / 4];
#pragma unroll
            for (int z = 0; z < ADAPTER_MAX_PARTS; ++z)
#pragma unroll
                for (int h = 0; h < KV / 4; ++h) w[z][h] = load16(t + min(z, p.parts - 1) * p.plane + 4 * h);
#pragma unroll
            for (int z = 0; z < ADAPTER_MAX_PARTS; ++z)
#pragma unroll
                for (int i = 0; i < KV; ++i)
                    sum[i] += z < p.parts && e0 + i < p.rank ? __uint_as_float(w[z][i / 4][i % 4]) : 0.0f;
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if constexpr (BF16) {
                const uint32_t w = f32x2_to_bf16x2_rne(sum[2 * d], sum[2 * d + 1]);
                const float a = sum[2 * d] - __uint_as_float(w << 16), b = sum[2 * d + 1] - __uint_as_float(w & 0xFFFF0000u);
                const float inf = __builtin_inff();   // which leaves nothing for the second term
                v[0][d] = w;
                v[PLANES - 1][d] = f32x2_to_bf16x2_rne(fabsf(a) < inf ? a : 0.0f, fabsf(b) < inf ? b : 0.0f);
            } else {
                v[0][d] = __float_as_uint(sum[d]);
            }
        }
    }
    // t of a row, if it `has` one.  PARTS: of parts, if there are.
    template <bool PARTS>
    static __device__ __forceinline__ void load_t(const AdapterArgs &p, bool has, int64_t row, int e0, u32x4 (&v)[PLANES])
    {
        if constexpr (PARTS) {
            if (p.parts > 0) {
                load_parts(p, has, row, e0, v);
                return;
            }
        }
        const In *t = static_cast<const In *>(p.t) + row * p.pitch + e0;
#pragma unroll
        for (int h = 0; h < PLANES; ++h) {
            v[h] = u32x4{0, 0, 0, 0};
            if (has && e0 < p.rank) v[h] = load16(t + h * p.plane);   // inside the pitch
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if constexpr (BF16)
                    v[h][d] &= e0 + 2 * d + 1 < p.rank ? 0xFFFFFFFFu : e0 + 2 * d < p.rank ? 0xFFFFu : 0u;
                else
                    v[h][d] = e0 + d < p.rank ? v[h][d] : 0u;
            }
        }
    }
};

// The numbers of a wave's rows in a tile, loaded before its product: row0: the first of
// the rows, rows: the end of those that there are.
template <class G>
struct TileAdapters {
    static constexpr int FR = G::BF16 ? 16 : 32;   // rows, or columns, of a fragment
    static constexpr bool PARTS = G::BM <= 64 && G::BN <= 64;
    int id[G::FN];

    __device__ __forceinline__ void load(const AdapterArgs &p, int lane, int row0, int rows)
    {
#pragma unroll
        for (int j = 0; j < G::FN; ++j) id[j] = p.ids[min(row0 + FR * j + lane % FR, rows - 1)];
    }

    // Adds the adapters to the wave's sums, STEPS steps of the rank at a time; col0: first
    // of the wave's columns, of N.  Slices of the summed axis take the adapters in turn.
    // What takes time are loads one after another, so those of t and of the first
    // adapters' b leave together, in smaller tiles, whose registers allow it, for two steps.
    // Large tiles' accumulators leave registers for one adapter's b.
    template <int STEPS, class Acc>
    __device__ __forceinline__ void add(const AdapterArgs &p, int lane, int row0, int rows, int col0, int N, int slice,
                                        int slices, Acc &acc) const
    {
        using Op = AdapterOperand<G::BF16>;
        using In = typename Op::In;
        constexpr int STEP = Op::KV * (64 / FR);           // k values of a step
        constexpr int BATCH = G::FM * G::FN > 16 ? 1 : 16 / G::FM / STEPS;   // adapters at a time
        const int c = lane % FR, q = lane / FR;
        uint32_t has = 0;                                  // bit j: this lane's row j has an adapter
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            if (row0 + FR * j + c < rows && (unsigned)id[j] < (unsigned)p.count) has |= 1u << j;
        if (__ballot(has != 0) == 0) return;
        for (int k0 = 0; k0 < p.rank; k0 += STEPS * STEP) {
            const bool whole = k0 + STEPS * STEP <= p.rank;   // of all lanes
            u32x4 t[STEPS][G::FN][Op::PLANES];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int k = k0 + s * STEP + q * Op::KV;
                if (whole && (!PARTS || p.parts == 0)) {
                    // rows without an adapter load what is there: it is not used
#pragma unroll
                    for (int j = 0; j < G::FN; ++j)
#pragma unroll
                        for (int h = 0; h < Op::PLANES; ++h)
                            t[s][j][h] = load16(static_cast<const In *>(p.t) +
                                                (int64_t)min(row0 + FR * j + c, rows - 1) * p.pitch + k + h * p.plane);
                } else {
#pragma unroll
                    for (int j = 0; j < G::FN; ++j) Op::template load_t<PARTS>(p, has >> j & 1, row0 + FR * j + c, k, t[s][j]);
                }
            }
            // Other adapters' rows must not see what one holds, and zeros for their t would make
            // NaN of its infinities.  So values of b that are not finite are left out, and in a
            // second turn their columns of the adapter's own rows become infinite, by products
            // of large numbers.  (Sums selected by row take the accumulators twice, which large
            // tiles have no registers for: 4096 rows of 8 requests, 4096 x 8192, rank 64: 765 us,
            // so 258.)
            bool finite = true;   // what this lane has read of the adapters
#pragma nounroll
            for (bool marked = false;; marked = true) {
                uint32_t left = has;
                int turn = 0;
                while (true) {
                    int e[BATCH];
#pragma unroll
                    for (int n = 0; n < BATCH; ++n) {
                        // the next adapter that is left, and this slice's
                        bool mine;
                        do {
                            e[n] = -1;
#pragma unroll
                            for (int j = G::FN - 1; j >= 0; --j) {
                                const uint64_t some = __ballot(left >> j & 1);
                                if (some != 0) e[n] = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(some));
                            }
#pragma unroll
                            for (int j = 0; j < G::FN; ++j)
                                if (id[j] == e[n]) left &= ~(1u << j);
                            mine = turn == slice;
                            turn = turn + 1 == slices ? 0 : turn + 1;
                        } while (e[n] >= 0 && !mine);
                    }
                    if (e[0] < 0) break;
                    u32x4 w[BATCH][STEPS][G::FM];
#pragma unroll
                    for (int n = 0; n < BATCH; ++n) {
                        if (e[n] < 0) break;
                        const In *b = static_cast<const In *>(p.b) + e[n] * p.stride_b;
#pragma unroll
                        for (int i = 0; i < G::FM; ++i) {
                            const In *row = b + (int64_t)min(col0 + FR * i + c, N - 1) * p.ldb + k0 + q * Op::KV;
#pragma unroll
                            for (int s = 0; s < STEPS; ++s)
                                w[n][s][i] = whole ? __builtin_bit_cast(u32x4, *reinterpret_cast<const typename Op::chunk *>(row + s * STEP))
                                                   : Op::load(row - k0 - q * Op::KV, k0 + s * STEP + q * Op::KV, p.rank);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < BATCH; ++n) {
                        if (e[n] < 0) break;
                        uint32_t exponents = 0;
#pragma unroll
                        for (int s = 0; s < STEPS; ++s)
#pragma unroll
                            for (int i = 0; i < G::FM; ++i) exponents = Op::largest(exponents, w[n][s][i]);
                        if (__ballot(Op::infinite(exponents)) != 0 || marked) {
                            finite = finite && !Op::infinite(exponents);
#pragma unroll
                            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                                for (int i = 0; i < G::FM; ++i) w[n][s][i] = Op::apart(w[n][s][i], marked);
                        }
#pragma unroll
                        for (int j = 0; j < G::FN; ++j) {
                            const bool mine = (has >> j & 1) && id[j] == e[n];
                            if (__ballot(mine) == 0) continue;
#pragma unroll
                            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                                for (int h = 0; h < Op::PLANES; ++h) {
                                    u32x4 v;
#pragma unroll
                                    for (int d = 0; d < 4; ++d) {
                                        v[d] = marked ? Op::LARGE : t[s][j][h][d];
                                        v[d] = mine ? v[d] : 0u;
                                    }
#pragma unroll
                                    for (int i = 0; i < G::FM; ++i) Op::mma(w[n][s][i], v, acc[i][j]);
                                }
                        }
                    }
                }
                if (marked || __ballot(!finite) == 0) break;
            }
        }
    }
};

// Without adapters: nothing.
struct NoAdapters {};

}  // namespace dg
