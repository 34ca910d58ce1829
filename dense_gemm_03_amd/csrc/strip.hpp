// A product's strip of a few rows whose weights are read once and hardly reused: waves
// stream them straight into registers (no LDS, no barrier in the loop), the next step's
// loads under way during this one's products, and their sums meet in LDS at the end.
#pragma once

#include "linear_kernel.hpp"

namespace dg {

// LDS accesses of this wave before and after stay in their order.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int lanes_below(uint64_t mask)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// A strip of output columns over k: P panels (gate and the other) of 16 W columns
// each, RT tiles of 16 rows of x, U steps per pass.  Lane (q, c) = (lane / 16, lane %
// 16) supplies KV values of k (16 bytes) of row c of a tile and of its column of w:
//   w as N x K (T): 16 bytes of row n0 + 16 f + c, fragment f;
//   w as K x N: KV loads of W consecutive columns n0 + W c .. of rows k .. k + KV - 1;
//     MFMA j has the columns n0 + W c + j.
// XP planes of x: bf16 as a sum of two, each multiplied.  Loads use the element's
// alignment, whatever the pitch.
template <bool BF16, bool T, int W, int P, int XP, int RT, int U>
struct Strip {
    using F = FewRows<BF16, T ? 1 : 0, W, 8>;   // its loads and products
    using In = typename F::In;
    static constexpr int KV = F::KV, STEP = 4 * KV, KP = U * STEP;
    struct Regs {
        u32x4 x[U][XP][RT];
        u32x4 w[T ? U * P * W : 1];
        uint32_t v[T ? 1 : U * P * KV][T ? 1 : F::PD];
    };

    const In *xr[RT];    // this lane's rows of x
    int64_t x_plane;     // elements from a plane to the next
    const In *w;         // the expert's weights: the same for all lanes, as n0 is,
    int64_t ldw;         // so that a load's address is a scalar and `off`
    uint32_t off[T ? W : KV];
    int q, c, n0, N, K;

    // First of this lane's columns (w as K x N): the last pieces of a strip that N
    // ends in move back to end with it, and repeat columns.
    __device__ __forceinline__ int first_col() const { return min(n0 + W * c, max(N - W, 0)); }

    // Lane, strip and extents; byte offsets stay below 2^32 (weights' pitch at most 2^24).
    __device__ __forceinline__ void place(int lane, int n0_, int N_, int K_, int64_t ldw_)
    {
        q = lane >> 4;
        c = lane & 15;
        n0 = n0_;
        N = N_;
        K = K_;
        ldw = ldw_;
        const uint32_t pitch = (uint32_t)ldw;
        if constexpr (T) {
#pragma unroll
            for (int f = 0; f < W; ++f)
                off[f] = ((uint32_t)(min(n0 + 16 * f + c, N - 1) - n0) * pitch + q * KV) * (uint32_t)sizeof(In);
        } else {
#pragma unroll
            for (int i = 0; i < KV; ++i) off[i] = ((q * KV + i) * pitch + first_col()) * (uint32_t)sizeof(In);
        }
    }

    // The pass at k0.  TAIL: K may end in it.  A lane whose values would pass the end
    // (K >= KV) loads the last KV values instead, and zeros in both operands for those
    // that a lower lane has: no branches.
    template <bool TAIL>
    __device__ __forceinline__ void load(int k0, Regs &r) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * STEP + q * KV;
            const int from = TAIL ? min(k, K - KV) : k, lost = k - from;   // values of a lane that do not count
            auto keep = [&](u32x4 v) {
                if constexpr (TAIL) {
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        if constexpr (BF16)
                            v[d] &= (2 * d >= lost ? 0xFFFFu : 0u) | (2 * d + 1 >= lost ? 0xFFFF0000u : 0u);
                        else
                            v[d] = d >= lost ? v[d] : 0u;
                    }
                }
                return v;
            };
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if constexpr (T) {
                    const unsigned char *base =
                        reinterpret_cast<const unsigned char *>(w + (int64_t)(p * N + n0) * ldw + k0) + u * STEP * sizeof(In);
#pragma unroll
                    for (int f = 0; f < W; ++f)
                        r.w[(u * P + p) * W + f] = keep(F::load_chunk(reinterpret_cast<const In *>(base + off[f]) - lost));
                } else {
                    const unsigned char *base =
                        reinterpret_cast<const unsigned char *>(w + (int64_t)(k0 + u * STEP) * ldw + p * (int64_t)N);
                    const In *row = w + from * ldw + p * (int64_t)N + first_col();   // of a tail
#pragma unroll
                    for (int i = 0; i < KV; ++i) {
                        union {
                            typename F::piece v;
                            uint32_t d[F::PD];
                        } t;
                        t.v = TAIL ? *reinterpret_cast<const typename F::piece *>(row + i * ldw)
                                   : *reinterpret_cast<const typename F::piece *>(base + off[i]);
#pragma unroll
                        for (int d = 0; d < F::PD; ++d)
                            r.v[(u * P + p) * KV + i][d] = !TAIL || i >= lost ? t.d[d] : 0u;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int h = 0; h < XP; ++h) r.x[u][h][t] = keep(F::load_chunk(xr[t] + h * x_plane + from));
        }
    }
    __device__ __forceinline__ void compute(const Regs &r, floatx4 (&acc)[P * W][RT]) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    u32x4 b;
                    if constexpr (T) {
                        b = r.w[(u * P + p) * W + j];
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int at = (u * P + p) * KV;
                            if constexpr (BF16)   // column j of two rows of k
                                b[i] = __builtin_amdgcn_perm(r.v[at + 2 * i + 1][j / 2], r.v[at + 2 * i][j / 2],
                                                             j & 1 ? 0x07060302u : 0x05040100u);
                            else
                                b[i] = r.v[at + i][j];
                        }
                    }
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int h = 0; h < XP; ++h) F::mma(r.x[u][h][t], b, acc[p * W + j][t]);
                }
    }
    // Column of the strip of this lane's sums of fragment j of a panel.
    __device__ __forceinline__ int column(int j) const { return T ? 16 * j + c : first_col() - n0 + j; }
};

template <int N, int RT>
__device__ __forceinline__ void clear(floatx4 (&acc)[N][RT])
{
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[j][t] = {0.0f, 0.0f, 0.0f, 0.0f};
}

// A strip of a product over the whole of k, for `count` rows of x (row(r): the place of
// the r-th); waves have a run of k each, and their sums meet in LDS: out(r, col, sums of
// the panels) for row r and column col of the strip.
//
// A wave goes round its run from a place that depends on the strip.  Rows of w as N x
// K often lie a power of two apart, and blocks in step would read from a few memory
// channels (16 tokens, 64 experts of 2048 x 1024: 129 us, in step 133).
template <int WV, bool BF16, bool T, int W, int P, int XP, int RT, int U, class Row, class Out>
__device__ __forceinline__ void product(const void *w, int64_t ldw, int N, int K, int n0, const void *x, int64_t x_plane,
                                        int count, Row &&row, float *sums, int lane, int wave, Out &&out)
{
    using S = Strip<BF16, T, W, P, XP, RT, U>;
    using In = typename S::In;
    constexpr int BN = 16 * W * P, ROWS = 16 * RT;
    S s;
    s.place(lane, n0, N, K, ldw);
    s.w = static_cast<const In *>(w);
    s.x_plane = x_plane;
#pragma unroll
    for (int t = 0; t < RT; ++t) s.xr[t] = static_cast<const In *>(x) + row(min(16 * t + s.c, count - 1));
    floatx4 acc[P * W][RT];
    clear(acc);
    typename S::Regs cur, nxt;
    const int passes = K / S::KP;   // whole ones; the cut one is the last wave's
    const int first = passes * wave / WV, mine = passes * (wave + 1) / WV - first;
    const bool tail = wave == WV - 1 && passes * S::KP < K;
    int at = mine > 0 ? n0 / (16 * W) % mine : 0;
    if (mine > 0) s.template load<false>((first + at) * S::KP, cur);
    for (int i = 1; i < mine; ++i) {
        at = at + 1 == mine ? 0 : at + 1;
        s.template load<false>((first + at) * S::KP, nxt);
        s.compute(cur, acc);
        cur = nxt;
    }
    if (tail) s.template load<true>(passes * S::KP, nxt);
    if (mine > 0) s.compute(cur, acc);
    if (tail) s.compute(nxt, acc);
    // half of the waves' sums, then the others' added to them: sums takes WV / 2 strips
    auto meet = [&](bool add) {
        float *mine = sums + wave % (WV / 2) * (ROWS * BN);
#pragma unroll
        for (int f = 0; f < P * W; ++f) {
            const int col = s.column(f % W);
            if (T || col >= W * s.c)   // (pieces that N's end moved back repeat columns of others)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float &at = mine[(16 * t + 4 * s.q + r) * BN + f / W * 16 * W + col];
                        at = add ? at + acc[f][t][r] : acc[f][t][r];
                    }
        }
        __syncthreads();
    };
    if (wave < WV / 2) meet(false);
    else __syncthreads();
    if (wave >= WV / 2) meet(true);
    else __syncthreads();
    for (int id = (int)threadIdx.x; id < count * 16 * W; id += 64 * WV) {
        const int r = id / (16 * W), col = id % (16 * W);
        if (n0 + col >= N) continue;
        float z[P];
#pragma unroll
        for (int f = 0; f < P; ++f) {
            z[f] = 0.0f;
#pragma unroll
            for (int v = 0; v < WV / 2; ++v) z[f] += sums[(v * ROWS + r) * BN + f * 16 * W + col];
        }
        out(r, col, z);
    }
}

}  // namespace dg
