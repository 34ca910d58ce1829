// Low-rank adapters in the linear layers' kernels: after a block's product its sums
// take up t . b^T, with t = scale x . a^T of the row's own adapter (adapter.hip forms
// it before the product).
//
// The ranks are a few k-steps more, so they cost the product little as MFMAs, but a
// tile may hold rows of several adapters: it goes through the adapters of its rows, each
// with the rows of t that are not its own as zeros.  Rows of a request lie together, so
// that is one or two adapters for most tiles.
//
// t is in fp32; bf16 products read it as a sum of two bf16 values (16 bits of it: two
// MFMAs instead of one, on the few steps that the ranks take).
#pragma once

#include "mma16.hpp"

namespace dg {

struct AdapterArgs {
    const float *t;         // parts x rows x pitch: sums over parts of k
    const void *b;          // per adapter N x rank
    const int32_t *ids;     // per row; outside 0 .. count-1: none
    int64_t ldb, stride_b;
    int64_t t_part;         // elements between parts
    int count, rank, pitch, parts;
};

// KV values of k from e0 of a row, zero from `end` on; loads at the element's alignment.
template <bool BF16>
struct AdapterOperand {
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    static constexpr int KV = BF16 ? 8 : 4;
    typedef In chunk __attribute__((ext_vector_type(KV), aligned(sizeof(In))));

    static __device__ __forceinline__ u32x4 load(const In *row, int e0, int end)
    {
        if (e0 + KV <= end) return __builtin_bit_cast(u32x4, *reinterpret_cast<const chunk *>(row + e0));
        union {
            u32x4 v;
            In e[KV];
        } u;
#pragma unroll
        for (int i = 0; i < KV; ++i) u.e[i] = e0 + i < end ? row[e0 + i] : In(0);
        return u.v;
    }
    // The same of t's row, where `mine`, in two terms (fp32: the first is all).
    static __device__ __forceinline__ void load_t(const AdapterArgs &p, bool mine, int64_t row, int e0, u32x4 &hi, u32x4 &lo)
    {
        float v[KV];
#pragma unroll
        for (int i = 0; i < KV; ++i) v[i] = 0.0f;
        if (mine && e0 < p.rank) {   // the pitch covers whole chunks
            for (int z = 0; z < p.parts; ++z) {
                const float *t = p.t + z * p.t_part + row * p.pitch + e0;
#pragma unroll
                for (int h = 0; h < KV; h += 4) {
                    const u32x4 w = load16(t + h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[h + i] += e0 + h + i < p.rank ? __uint_as_float(w[i]) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if constexpr (BF16) {
                const uint32_t w = f32x2_to_bf16x2_rne(v[2 * d], v[2 * d + 1]);
                const float r0 = v[2 * d] - __uint_as_float(w << 16), r1 = v[2 * d + 1] - __uint_as_float(w & 0xFFFF0000u);
                const float inf = __builtin_inff();   // which leaves nothing for the second term
                hi[d] = w;
                lo[d] = f32x2_to_bf16x2_rne(fabsf(r0) < inf ? r0 : 0.0f, fabsf(r1) < inf ? r1 : 0.0f);
            } else {
                hi[d] = __float_as_uint(v[d]);
                lo[d] = 0;
            }
        }
    }
};

__device__ __forceinline__ int adapter_of_row(const AdapterArgs &p, int64_t row)
{
    const int id = p.ids[row];
    return (unsigned)id < (unsigned)p.count ? id : -1;
}

// Adds the adapters of a tile's rows to a wave's sums.  row0: first of the wave's rows,
// rows: the end of those that there are; col0: first of its columns, of N.
template <class G, class Acc>
__device__ __forceinline__ void add_adapters(const AdapterArgs &p, int lane, int row0, int rows, int col0, int N, Acc &acc)
{
    using Op = AdapterOperand<G::BF16>;
    using In = typename Op::In;
    constexpr int FR = G::BF16 ? 16 : 32;              // rows, or columns, of a fragment
    constexpr int STEP = Op::KV * (64 / FR);           // k values of a step
    const int c = lane % FR, q = lane / FR;
    int id[G::FN];
#pragma unroll
    for (int j = 0; j < G::FN; ++j) {
        const int row = row0 + FR * j + c;
        id[j] = row < rows ? adapter_of_row(p, row) : -1;
    }
    while (true) {
        int e = -1;   // the first adapter that is left
#pragma unroll
        for (int j = G::FN - 1; j >= 0; --j) {
            const uint64_t left = __ballot(id[j] >= 0);
            if (left != 0) e = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(left));
        }
        if (e < 0) return;
        const In *b = static_cast<const In *>(p.b) + e * p.stride_b;
        for (int k0 = 0; k0 < p.rank; k0 += STEP) {
            const int k = k0 + q * Op::KV;
            u32x4 w[G::FM];
#pragma unroll
            for (int i = 0; i < G::FM; ++i) w[i] = Op::load(b + (int64_t)min(col0 + FR * i + c, N - 1) * p.ldb, k, p.rank);
#pragma unroll
            for (int j = 0; j < G::FN; ++j) {
                if (__ballot(id[j] == e) == 0) continue;
                u32x4 hi, lo;
                Op::load_t(p, id[j] == e, row0 + FR * j + c, k, hi, lo);
#pragma unroll
                for (int i = 0; i < G::FM; ++i) {
                    if constexpr (G::BF16) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, w[i]), __builtin_bit_cast(bf16x8, hi), acc[i][j], 0, 0, 0);
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, w[i]), __builtin_bit_cast(bf16x8, lo), acc[i][j], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                __uint_as_float(w[i][d]), __uint_as_float(hi[d]), acc[i][j], 0, 0, 0);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            if (id[j] == e) id[j] = -1;
    }
}

}  // namespace dg
