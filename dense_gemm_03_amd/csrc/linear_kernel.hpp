// Device code of the linear layers: the tiled product of gemm_kernel.hpp with
// row groups and an epilogue of its own.
//
//     y = act(alpha x . w + bias) + residual               (x k-contiguous)
//     dw = alpha x^T . dz + beta dw                        (x outer-contiguous)
//
// In the first form the groups cut the rows of the output: a group's rows are
// covered by tiles of BM rows of their own, so a tile never mixes two weight
// matrices, and the tile list is worked out on the device from the offsets
// (GroupRows).  In the second the groups cut the summed axis: every group has
// an output matrix, and its blocks walk that group's rows only.
#pragma once

#include "linear_pieces.hpp"
#include "mma16.hpp"

namespace dg {

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// What becomes of the sums: the operands of the epilogue.
struct EpilogueArgs {
    void *C;                // y, or dw
    void *pre;              // receives z; or nullptr
    const void *residual;   // nullptr: none (dw: dw itself when beta != 0)
    const void *bias;       // nullptr: none
    int64_t ldc, ldr, ldp;
    float alpha, beta;      // beta scales the residual
    int act;
    int out_bf16, bias_bf16;
    int vec;                // rows of C, pre and residual are 16-byte aligned
};

struct LinearArgs {
    const void *x, *w;      // x and w; of the second form, x and dz (or, for dw^T, dz and x)
    const int32_t *offsets; // nullptr: one group of all rows
    float *ws;              // partial sums of `splits` > 1 slices
    EpilogueArgs e;
    int64_t ldx, ldw;
    int64_t stride_w;       // elements between the groups' w (first form)
    int64_t stride_c;       // elements between the groups' dw (second form)
    int64_t stride_bias;
    int rows;               // rows of x: M of the first form, K of the second
    int M, N, K;            // extents of one group's product; the first form's M and the
                            // second's K are replaced by the group's row count
    int m_load, n_load;     // outer extents that the loads may read, as KernelArgs
    int groups;             // at least 1
    int tiles_m, tiles_n;   // tiles_m: second form only
    int splits, k_per_split;
    int group_m;
    int direct_ok;
    int slots;              // compute units per XCD (for entries of one block per unit)
};

// ------------------------------------------------------------- activations --

// sigmoid(x) = 1 / (1 + e^-x), with the hardware's exp2 and reciprocal (1 ulp
// each; the product x log2(e) adds |x| 2^-24 relative).  e^-x overflows to
// infinity for x below -88.7 and the reciprocal of it is 0.
__device__ __forceinline__ float sigmoid(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// 2 sqrt(2/pi): gelu_tanh(z) = z (1 + tanh(u / 2)) / 2 = z sigmoid(u),
// u = 2 sqrt(2/pi) (z + 0.044715 z^3).
constexpr float kGeluA = 1.5957691216057308f;
constexpr float kGeluB = 1.5957691216057308f * 0.044715f;

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2) with it.  Phi(-|z|)
// is e times a polynomial of degree 9 in t = 1 / (1 + 0.28 |z|), off by 9e-8 of itself
// up to |z| = 40; where |z| < 1, 1/2 + z Q(z^2) with Q of degree 5 is off by 1e-9.
// Both were fitted to the functions in double precision for the least relative
// error.  In fp32 z Phi(z) is off by 2.7e-7 of itself for z > -1, by 7e-7 for z > -3
// and, with the exponent's rounding, by 3e-6 for z > -8.  Without Q (NEAR false) Phi
// is off by 5e-7 of itself for |z| < 1.
template <bool NEAR>
__device__ __forceinline__ float normal_cdf(float z, float &e)
{
    const float s = z * z;
    e = __builtin_amdgcn_exp2f(-0.72134752f * s);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, fabsf(z), 1.0f));
    float g = __builtin_fmaf(t, 0.0258585084f, -0.0980442613f);
    g = __builtin_fmaf(t, g, 0.0995351374f);
    g = __builtin_fmaf(t, g, -0.0124129951f);
    g = __builtin_fmaf(t, g, 0.0755921081f);
    g = __builtin_fmaf(t, g, 0.0828876942f);
    g = __builtin_fmaf(t, g, 0.103185914f);
    g = __builtin_fmaf(t, g, 0.111694008f);
    g = __builtin_fmaf(t, g, 0.111703925f);
    const float tail = t * g * e;
    const float far = z > 0.0f ? 1.0f - tail : tail;
    if constexpr (!NEAR) return far;
    float q = __builtin_fmaf(s, -7.65420828e-06f, 0.000113486371f);
    q = __builtin_fmaf(s, q, -0.00118632999f);
    q = __builtin_fmaf(s, q, 0.00997332297f);
    q = __builtin_fmaf(s, q, -0.0664903596f);
    q = __builtin_fmaf(s, q, 0.398942292f);
    return s < 1.0f ? __builtin_fmaf(z, q, 0.5f) : far;
}

// The same for results that become bf16, half a step of which is 3.9e-3: a
// polynomial of degree 7, off by 2.2e-6 (bf16 gelu layer of 4096 x 4096 x 512: 32.9
// us; 34.0 with the form above).
__device__ __forceinline__ float normal_cdf_bf16(float z)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.275f, fabsf(z), 1.0f));
    float g = __builtin_fmaf(t, -0.0552612655f, 0.129859015f);
    g = __builtin_fmaf(t, g, 0.00389020261f);
    g = __builtin_fmaf(t, g, 0.103644535f);
    g = __builtin_fmaf(t, g, 0.0981924906f);
    g = __builtin_fmaf(t, g, 0.109972589f);
    g = __builtin_fmaf(t, g, 0.109701321f);
    const float tail = t * g * __builtin_amdgcn_exp2f(-0.72134752f * z * z);
    return z > 0.0f ? 1.0f - tail : tail;
}

// act(z) of V values that become bf16 or fp32, the activation chosen once for
// all of them.  Both forms with a sigmoid are z sigmoid(z (a + b z^2)); a NaN
// stays a NaN.
template <int V>
__device__ __forceinline__ void act_apply(int act, bool bf16, float (&v)[V])
{
    if (act == ACT_NONE) return;
    if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] <= 0.0f ? 0.0f : v[i];
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float e;
            v[i] *= bf16 ? normal_cdf_bf16(v[i]) : normal_cdf<true>(v[i], e);
        }
    } else {
        const float a = act == ACT_SILU ? 1.0f : kGeluA, b = act == ACT_SILU ? 0.0f : kGeluB;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid(v[i] * __builtin_fmaf(b * v[i], v[i], a));
    }
}

// act'(z), written over z.  Beyond |z| = 100 every slope here is 0 or 1 to
// more digits than fp32 holds; the bound keeps its products of a vanishing
// and a growing factor from forming 0 x infinity.  A NaN stays.  FINE: for a dz in
// fp32 (dbias sums fp32 values for either).
template <int V, bool FINE>
__device__ __forceinline__ void act_slope(int act, float (&v)[V])
{
    auto bounded = [](float z) { return z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z; };
    if (act == ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] > 0.0f ? 1.0f : v[i] <= 0.0f ? 0.0f : v[i];
    } else if (act == ACT_GELU) {   // Phi(z) + z phi(z)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = bounded(v[i]);
            float e;
            const float cdf = normal_cdf<FINE>(z, e);
            v[i] = cdf + z * 0.39894228f * e;
        }
    } else {                        // q + z q (1 - q) u',  q = sigmoid(u), u = z (a + b z^2)
        const float a = act == ACT_SILU ? 1.0f : kGeluA, b = act == ACT_SILU ? 0.0f : kGeluB;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = bounded(v[i]), bz = b * z;
            const float q = sigmoid(z * __builtin_fmaf(bz, z, a));
            v[i] = __builtin_fmaf(z * q * (1.0f - q), __builtin_fmaf(3.0f * bz, z, a), q);
        }
    }
}

// ------------------------------------------------------------ row groups ----

__device__ __forceinline__ int clamp_row(int o, int rows) { return o < 0 ? 0 : o > rows ? rows : o; }

// First row and row count of group g, whatever offsets holds: inside 0 .. rows.
__device__ __forceinline__ void group_span(const int32_t *offsets, int g, int rows, int &lo, int &m)
{
    if (offsets == nullptr) {
        lo = 0;
        m = rows;
        return;
    }
    lo = clamp_row(offsets[g], rows);
    const int hi = clamp_row(offsets[g + 1], rows);
    m = hi > lo ? hi - lo : 0;
}

// The list of row tiles of `bm` rows over all groups, from the offsets: each
// wave forms it for itself, 64 groups at a time (one per lane, a scan across
// the lanes), so no launch before this one and no memory is needed.  With
// `half` > 0 a group's last tile of at most that many rows is small, and the
// small tiles form a list of their own behind the others.
//
// Offsets that fall can claim the same rows many times over.  Sums stop at CAP,
// beyond any that offsets in order can have, and the lists at what those can
// have: the grid, the workspaces and 32-bit products of either are made for that.
struct GroupRows {
    static constexpr int CAP = (1 << 30) - 1;
    int total, small;   // tiles of all groups: all but the small ones, the small ones

    __device__ __forceinline__ static int lane_tiles(const int32_t *offsets, int g, int groups,
                                                     int rows, int bm, int half, bool want_small,
                                                     int &lo, int &m)
    {
        lo = 0;
        m = 0;
        if (g < groups) group_span(offsets, g, rows, lo, m);
        const int rest = m % bm;
        const bool is_small = rest > 0 && rest <= half;
        return want_small ? (is_small ? 1 : 0) : m / bm + (rest > half ? 1 : 0);
    }
    __device__ __forceinline__ static int scan(int v, int lane)
    {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(v, d);
            if (lane >= d) v = min(v + o, CAP);
        }
        return v;
    }
    __device__ __forceinline__ GroupRows(const int32_t *offsets, int groups, int rows, int bm, int lane,
                                         int half = 0)
    {
        total = small = 0;
        if (offsets == nullptr) {
            const int rest = rows % bm;
            small = rest > 0 && rest <= half ? 1 : 0;
            total = rows / bm + (rest > half ? 1 : 0);
            return;
        }
        for (int base = 0; base < groups; base += 64) {
            int lo, m;
            const int t = lane_tiles(offsets, base + lane, groups, rows, bm, half, false, lo, m);
            total = min(total + __builtin_amdgcn_readlane(scan(t, lane), 63), CAP);
            if (half > 0)
                small += __builtin_popcountll(__ballot(m % bm > 0 && m % bm <= half));
        }
        total = min(total, rows / bm + min(groups, rows));
        small = min(small, min(groups, rows));
    }
    // Group, its first row, its rows and the tile inside it of tile `t` of
    // either list.
    __device__ __forceinline__ void find(const int32_t *offsets, int groups, int rows, int bm,
                                         int lane, int half, bool want_small, int t, int &group, int &lo,
                                         int &m, int &tm) const
    {
        group = 0;
        lo = 0;
        m = rows;
        tm = want_small ? rows / bm : t;
        if (offsets == nullptr) return;
        int before = 0;
        for (int base = 0; base < groups; base += 64) {
            int l, n;
            const int mine = lane_tiles(offsets, base + lane, groups, rows, bm, half, want_small, l, n);
            const int upto = before + scan(mine, lane);
            const uint64_t past = __ballot(upto > t);
            if (past != 0) {
                const int at = __builtin_ctzll(past);
                group = base + at;
                lo = __builtin_amdgcn_readlane(l, at);
                m = __builtin_amdgcn_readlane(n, at);
                tm = want_small ? m / bm
                                : t - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(mine, at));
                return;
            }
            before = min(__builtin_amdgcn_readlane(upto, 63), CAP);
        }
    }
};

// Place of this block among `active` blocks, or -1: consecutive places run on
// one XCD (the hardware deals workgroups to the 8 XCDs in turn).  The grid is
// a multiple of 8 and at least `active` rounded up to one; unlike a cut of the
// whole grid, this spreads the blocks that have work evenly over the XCDs when
// the grid is only an upper bound.
__device__ __forceinline__ int xcd_place(int active)
{
    const int bid = (int)blockIdx.x, per = (active + 7) >> 3;
    const int at = (bid & 7) * per + (bid >> 3);
    return (bid >> 3) < per && at < active ? at : -1;
}

// Group of rank o in the order of falling row counts (ties: the lower group
// first), for up to 64 groups, one per lane; the groups as they are for more.
// Blocks of the largest groups start first, so that none of them runs alone at
// the end.
__device__ __forceinline__ int group_of_rank(const int32_t *offsets, int groups, int rows, int lane, int o)
{
    if (offsets == nullptr || groups == 1 || groups > 64) return o;
    int lo, m = -1;
    if (lane < groups) group_span(offsets, lane, rows, lo, m);
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const int other = __builtin_amdgcn_readlane(m, g);
        rank += other > m || (other == m && g < lane) ? 1 : 0;
    }
    return __builtin_ctzll(__ballot(lane < groups && rank == o));
}

// --------------------------------------------------------------- epilogue --

// V values of an output row from element idx on, n of them inside the matrix.
// WHOLE: all of them, 16 bytes at a 16-byte boundary; else decided here.
template <int V, bool WHOLE = false>
__device__ __forceinline__ void load_out(const void *C, int64_t idx, int n, bool bf16, bool vec,
                                         float (&v)[V])
{
    if (V == 8 && bf16) {
        const uint16_t *c = static_cast<const uint16_t *>(C) + idx;
        if (WHOLE || (vec && n >= V)) {
            const u32x4 w = load16(c);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                v[2 * i] = __uint_as_float(w[i & 3] << 16);
                v[2 * i + 1] = __uint_as_float(w[i & 3] & 0xFFFF0000u);
            }
            return;
        }
    }
    if (V == 4 && bf16 && !WHOLE && vec && n >= V) {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(C) + idx);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i & 1] << 16);
            v[2 * i + 1] = __uint_as_float(w[i & 1] & 0xFFFF0000u);
        }
        return;
    }
    if (V == 4 && !bf16) {
        const float *c = static_cast<const float *>(C) + idx;
        if (WHOLE || (vec && n >= V)) {
            const u32x4 w = load16(c);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i & 3]);
            return;
        }
    }
    if constexpr (!WHOLE) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = i >= n ? 0.0f
                   : bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(C)[idx + i] << 16)
                          : static_cast<const float *>(C)[idx + i];
    }
}

// Rounded once, to nearest even (bf16), or as they are.  Non-temporal: the
// layer's outputs are written once and must not evict the operand tiles that
// other blocks still stream.
template <int V, bool WHOLE = false>
__device__ __forceinline__ void store_outs(void *C, int64_t idx, int n, bool bf16, bool vec,
                                           const float (&v)[V])
{
    if (V == 8 && bf16 && (WHOLE || (vec && n >= V))) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i & 3] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(C) + idx));
        return;
    }
    if (V == 4 && bf16 && !WHOLE && vec && n >= V) {
        u32x2 w;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i & 1] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(C) + idx) = w;
        return;
    }
    if (V == 4 && !bf16 && (WHOLE || (vec && n >= V))) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < V; ++i) w[i & 3] = __float_as_uint(v[i]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(static_cast<float *>(C) + idx));
        return;
    }
    if constexpr (!WHOLE) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i >= n) break;
            if (bf16)
                static_cast<uint16_t *>(C)[idx + i] = f32_to_bf16_rne(v[i]);
            else
                static_cast<float *>(C)[idx + i] = v[i];
        }
    }
}

// The bias of columns col .. col + V - 1 of group g (zeros where there is none).
template <int V>
__device__ __forceinline__ void load_bias(const EpilogueArgs &e, int64_t at, int n, float (&b)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.0f;
    if (e.bias == nullptr) return;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (i < n)
            b[i] = e.bias_bf16
                       ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(e.bias)[at + i] << 16)
                       : static_cast<const float *>(e.bias)[at + i];
}

// V sums of one output row from column col on, n of them inside the matrix,
// finished and stored.  `row` counts rows of C, pre and residual; c_off is an
// element offset of C (the group's dw).
template <int V, bool WHOLE = false>
__device__ __forceinline__ void finish_piece(const EpilogueArgs &e, int64_t c_off, int64_t row,
                                             int col, int n, const float (&bias)[V], float (&v)[V])
{
    // pieces of 8 are of bf16 outputs only
    const bool bf16 = V == 8 || (WHOLE ? false : e.out_bf16 != 0), vec = e.vec != 0;
    float old[V];
    if (e.residual != nullptr) load_out<V, WHOLE>(e.residual, c_off + row * e.ldr + col, n, bf16, vec, old);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e.alpha * v[i] + bias[i];
    if (e.pre != nullptr) store_outs<V, WHOLE>(e.pre, row * e.ldp + col, n, bf16, vec, v);
    act_apply<V>(e.act, bf16, v);
    if (e.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += e.beta * old[i];
    }
    store_outs<V, WHOLE>(e.C, c_off + row * e.ldc + col, n, bf16, vec, v);
}

// The block's accumulators as pieces of V consecutive columns of an output row
// per lane: out(row, col, piece) for each, row and col inside the block.
//
// The products run with w (or dz) as the first operand, so a lane's four
// consecutive accumulators are four consecutive columns of one output row.
// Each wave passes them through LDS, its share of the stages (free after the
// main loop), as many rows at a time as fit: 16-byte writes, then a loop in
// which the wave reads whole rows, 16 bytes of output per lane.  The loop holds
// the epilogue's code once; written out for every accumulator instead, without
// LDS, it filled the instruction cache and spilled registers.  The 16-byte
// chunks of a row are permuted by its number, so that the lanes of a write (16
// or 32 rows at the same columns) spread over the banks.
template <class G, int V>
struct StagedTile {
    static constexpr int COLS = G::WTM;
    static constexpr int FR = G::BF16 ? 16 : 32;    // rows of a fragment
    // rows that fit a wave's share, whole fragments, a divisor of its rows
    static constexpr int SHARE = G::STAGE_BYTES * 2 / G::NW;   // of two stages
    static constexpr int FIT = SHARE / (COLS * 4);
    static constexpr int ROWS = FIT >= G::WTN ? G::WTN : FIT >= G::WTN / 2 ? G::WTN / 2 : 32;
    static_assert(ROWS * COLS * 4 <= SHARE && G::WTN % ROWS == 0 && ROWS % FR == 0, "whole fragments fit");
    static constexpr int CPR = COLS / V, PASSES = ROWS * CPR / 64;
    static_assert(ROWS * CPR % 64 == 0, "whole passes");
    static __device__ __forceinline__ int place(int row, int col)
    {
        return row * COLS + (col ^ ((row << 2) & (COLS - 4)));
    }
    // The share of wave `wv`: half the waves in either of the first two stages.
    static __device__ __forceinline__ unsigned char *share(unsigned char *s0, unsigned char *s1, int wv)
    {
        constexpr int HALF = G::NW > 1 ? G::NW / 2 : 1;
        return (wv < HALF ? s0 : s1) + (wv % HALF) * (ROWS * COLS * 4);
    }
    template <class Acc, class Out>
    static __device__ __forceinline__ void run(unsigned char *scr, const BlockCtx<G> &c, const Acc &acc,
                                               Out &&out)
    {
        static_for<0, G::WTN / ROWS>([&](auto s_c) {
            constexpr int slab = decltype(s_c)::value;
            static_for<0, ROWS / FR>([&](auto j_c) {
                constexpr int j = decltype(j_c)::value;
                static_for<0, G::FM>([&](auto i_c) {
                    constexpr int i = decltype(i_c)::value;
                    if constexpr (G::BF16) {
                        *reinterpret_cast<floatx4 *>(
                            scr + 4 * place(16 * j + (c.lane & 15), 16 * i + 4 * (c.lane >> 4))) =
                            acc[i][slab * (ROWS / FR) + j];
                    } else {
                        const floatx16 &a = acc[i][slab * (ROWS / FR) + j];
                        static_for<0, 4>([&](auto g_c) {
                            constexpr int g = 4 * decltype(g_c)::value;
                            *reinterpret_cast<floatx4 *>(
                                scr + 4 * place(32 * j + (c.lane & 31), 32 * i + 2 * g + 4 * (c.lane >> 5))) =
                                floatx4{a[g], a[g + 1], a[g + 2], a[g + 3]};
                        });
                    }
                });
            });
            // a wave's LDS accesses complete in order: the reads see the
            // writes above, and the next slab's writes follow these reads
#pragma unroll 2
            for (int u = 0; u < PASSES; ++u) {
                const int ch = c.lane + 64 * u, row = ch / CPR, col = ch % CPR * V;
                float v[V];
#pragma unroll
                for (int h = 0; h < V; h += 4) {
                    const u32x4 w = lds_load16(scr, 4 * place(row, col + h));
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[h + i] = __uint_as_float(w[i]);
                }
                out(c.wcol * G::WTN + ROWS * slab + row, c.wrow * G::WTM + col, v);
            }
        });
    }
};

// ------------------------------------------------------------------ kernel --

// Global -> registers of one operand's k-tile at k0 with masks, rows 16-byte
// aligned: a chunk that holds an element of the matrix is read whole (it lies
// inside the row's pitch or on the page of the row's last element), the
// elements from kend on are zeros.  n_outer is a whole number of chunks where
// it runs along the rows.
template <class T>
__device__ __forceinline__ void load_tile_chunks(const typename T::In *X, int64_t ld, int outer0, int n_outer,
                                                 int k0, int kend, int tid, u32x4 (&r)[T::PER_THREAD])
{
#pragma unroll
    for (int u = 0; u < T::PER_THREAD; ++u) {
        const int ch = tid + u * T::NT;
        const int row = ch / T::CPR, e = (ch % T::CPR) * T::VEC;
        if constexpr (T::LAYOUT == KMAJOR) {
            const int left = kend - k0 - e;   // elements of the chunk before kend
            u32x4 v = {0, 0, 0, 0};
            if (outer0 + row < n_outer && left > 0) v = load16(X + (int64_t)(outer0 + row) * ld + k0 + e);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if constexpr (T::ES == 4)
                    v[d] = d < left ? v[d] : 0u;
                else
                    v[d] &= 2 * d + 1 < left ? 0xFFFFFFFFu : 2 * d < left ? 0xFFFFu : 0u;
            }
            r[u] = v;
        } else {
            r[u] = u32x4{0, 0, 0, 0};
            if (k0 + row < kend && outer0 + e < n_outer) r[u] = load16(X + (int64_t)(k0 + row) * ld + outer0 + e);
        }
    }
}

// The output tile of a block: rows row0 .. of the group's output (its m rows,
// or the M rows of dw), columns col0 .. .
struct TileSpec {
    int slice, group;
    int lo, m;          // the group's first row and rows
    int row0, col0;
};

// One block's tile, all of it: main loop and epilogue.  The main loops' first
// operand is w (or dz), whose rows are output columns, the second x, whose rows
// are output rows: G is the geometry of the transposed tile.  The stages are
// the kernel's arrays, at least as large as G's.
template <class G, bool ALIGNED>
__device__ __forceinline__ void linear_tile(const LinearArgs &p, const TileSpec &t, unsigned char *lds0,
                                            unsigned char *lds1, unsigned char *lds2, unsigned char *lds3)
{
    using In = typename G::In;
    constexpr bool BF16 = G::BF16, WGRAD = G::LB == MNMAJOR;   // groups cut the summed axis
    constexpr int BM = G::BN, BN = G::BM, BK = G::BK;
    using Sum = typename std::conditional<BF16, floatx4, floatx16>::type;
    constexpr int SUMS = BF16 ? 4 : 16;
    constexpr bool PINNED = BF16 && G::NW == 4 && BK == 64 && G::STAGES == 2 && ALIGNED;

    BlockCtx<G> c;
    c.tid = (int)threadIdx.x;
    c.lane = c.tid & 63;
    const int wave = c.tid >> 6;
    c.wrow = wave / G::WN;
    c.wcol = wave % G::WN;
    c.bm = t.col0;
    c.bn = t.row0;
    c.lda = p.ldw;
    c.ldb = p.ldx;
    c.B = static_cast<const In *>(p.x) + (int64_t)t.lo * p.ldx;
    c.M = p.n_load;
    int K, kps;
    if constexpr (WGRAD) {
        c.A = static_cast<const In *>(p.w) + (int64_t)t.lo * p.ldw;
        c.N = p.m_load;
        K = t.m;
        // whole k-tiles per slice; a slice past the group's rows sums nothing
        kps = ((K + BK - 1) / BK + p.splits - 1) / p.splits * BK;
    } else {
        c.A = static_cast<const In *>(p.w) + t.group * p.stride_w;
        c.N = t.m;
        K = p.K;
        kps = p.k_per_split;
    }
    const int kbeg = min(K, t.slice * kps);
    c.kend = min(K, kbeg + kps);
    const int ntiles = (c.kend - kbeg + BK - 1) / BK;

    Sum acc[G::FM][G::FN];
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < G::FN; ++fn)
#pragma unroll
            for (int r = 0; r < SUMS; ++r) acc[fm][fn][r] = 0.0f;

    // The choice between the loops is that of the dense product, on the
    // group's rows: whole k-tiles through direct loads of 16 bytes per lane
    // (aligned rows) or 4 range-checked ones, the rest masked.
    {
        const bool edge_mn = c.bm + BN > c.M || c.bn + BM > c.N;
        const bool edge16 = (G::LA == KMAJOR || c.M % G::VEC == 0) &&
                            (G::LB == KMAJOR || c.N % G::VEC == 0);
        const bool x4 = ALIGNED && p.direct_ok && (!edge_mn || edge16);
        const bool pairs_ok =
            !BF16 || (((p.ldw | p.ldx) & 1) == 0 && (((uintptr_t)c.A | (uintptr_t)c.B) & 3) == 0 &&
                      (G::LA == KMAJOR || (c.M & 1) == 0) && (G::LB == KMAJOR || (c.N & 1) == 0));
        const bool dw = G::DMA4 && !PINNED && p.direct_ok && pairs_ok && !x4;
        const int nfast = x4 || dw ? (c.kend - kbeg) / BK : 0;
        // Blocks of different groups start at different k-tiles.  Weights whose
        // rows lie a power of two apart keep their k-tile on a few memory
        // channels, and blocks in step would all read from those (16 groups of
        // 512 rows, N x K weights of 4096 x 4096: 264 -> 232 us); blocks that
        // share weights or rows are of one group and stay in step.
        c.rot = WGRAD ? 0 : 8 * t.group;
        if constexpr (G::DMA4 && !PINNED) {
            c.a_end = operand_end_bytes<typename G::TA>(p.ldw, c.M, K);
            c.b_end = operand_end_bytes<typename G::TB>(p.ldx, c.N, K);
            if (dw && nfast > 0) {
                if constexpr (BF16)
                    main_loop16_direct<G, 4>(lds0, lds1, lds2, lds3, c, kbeg, nfast, acc);
                else
                    main_loop_direct<G, 4>(lds0, lds1, lds2, lds3, c, kbeg, nfast, acc);
            }
        }
        if constexpr (ALIGNED) {
            if (x4 && nfast > 0) {
                if constexpr (PINNED)
                    main_loop_pinned<G>(lds0, lds1, c, kbeg, nfast, acc);
                else if constexpr (BF16)
                    main_loop16_direct<G, 16>(lds0, lds1, lds2, lds3, c, kbeg, nfast, acc);
                else
                    main_loop_direct<G, 16>(lds0, lds1, lds2, lds3, c, kbeg, nfast, acc);
            }
        }
        if (ntiles > nfast) {
            auto load = [&](int k0, StageRegs<G> &r) {
                if constexpr (ALIGNED) {
                    load_tile_chunks<typename G::TA>(c.A, c.lda, c.bm, c.M, k0, c.kend, c.tid, r.a);
                    load_tile_chunks<typename G::TB>(c.B, c.ldb, c.bn, c.N, k0, c.kend, c.tid, r.b);
                } else {
                    global_load_masked<false>(c, k0, r);
                }
            };
            if constexpr (BF16)
                main_loop16_masked(lds0, lds1, c, kbeg + nfast * BK, ntiles - nfast, acc, load);
            else
                main_loop_masked(lds0, lds1, c, kbeg + nfast * BK, ntiles - nfast, acc, load);
        }
    }

    const int out_rows = WGRAD ? p.M : t.m;   // rows of this group's output
    // the last readers of the stages have passed a barrier
    unsigned char *scr = StagedTile<G, 4>::share(lds0, lds1, __builtin_amdgcn_readfirstlane(wave));
    if (p.splits > 1) {
        // raw sums, summed by the reduce kernel: slice-major, first form rows x
        // N by global row, second form groups x M x N
        const int64_t first = WGRAD ? ((int64_t)t.slice * p.groups + t.group) * p.M
                                    : (int64_t)t.slice * p.rows + t.lo;
        float *out = p.ws + (first + t.row0) * p.N + t.col0;
        const bool quads = (p.N & 3) == 0;
        StagedTile<G, 4>::run(scr, c, acc, [&](int r, int cc, float (&v)[4]) {
            const int n = p.N - t.col0 - cc;
            if (t.row0 + r >= out_rows || n <= 0) return;
            float *o = out + (int64_t)r * p.N + cc;
            if (quads) {
                *reinterpret_cast<u32x4 *>(o) = __builtin_bit_cast(u32x4, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < n) o[i] = v[i];
            }
        });
        return;
    }
    const int64_t crow0 = (WGRAD ? 0 : t.lo) + t.row0;
    const int64_t c_off = WGRAD ? t.group * p.stride_c : 0;
    const int64_t bias0 = t.group * p.stride_bias + t.col0;
    auto finish = [&](auto v_c) {
        constexpr int V = decltype(v_c)::value;
        using S = StagedTile<G, V>;
        // a lane's columns are the same in every piece: 64 lanes take whole rows
        static_assert(64 % S::CPR == 0, "whole rows per pass");
        const int cc = c.wrow * G::WTM + c.lane % S::CPR * V, n = p.N - t.col0 - cc;
        const int rows = out_rows - t.row0;
        float bias[V];
        load_bias<V>(p.e, bias0 + cc, n, bias);
        if (t.col0 + BN <= p.N && p.e.vec) {
            S::run(scr, c, acc, [&](int r, int, float (&v)[V]) {
                if (r < rows) finish_piece<V, true>(p.e, c_off, crow0 + r, t.col0 + cc, V, bias, v);
            });
        } else {
            S::run(scr, c, acc, [&](int r, int, float (&v)[V]) {
                if (r < rows && n > 0) finish_piece<V, false>(p.e, c_off, crow0 + r, t.col0 + cc, n, bias, v);
            });
        }
    };
    if (p.e.out_bf16)
        finish(std::integral_constant<int, 8>());
    else
        finish(std::integral_constant<int, 4>());
}

// BM x BN output tile, WM x WN waves; LX and LW: how x and w (dz) lie in memory.
template <bool BF16, int BM, int BN, int BK, int WM, int WN, int STAGES, int LX, int LW, bool ALIGNED>
__global__ void __launch_bounds__(64 * WM * WN) linear_kernel(LinearArgs p)
{
    using G = typename std::conditional<BF16, Geo16<BN, BM, BK, WN, WM, STAGES, LW, LX>,
                                        Geo<BF16, BN, BM, BK, WN, WM, STAGES, LW, LX>>::type;
    constexpr bool WGRAD = LX == MNMAJOR;
    // one block per compute unit, and pieces of a tile to choose from
    constexpr bool PIECES = BF16 && BM == 256 && BN == 256 && WM * WN == 4;

    // pieces divide one array in ways of their own
    __shared__ __attribute__((aligned(1024))) unsigned char all[PIECES ? 9 * G::STAGE_BYTES / 4 : 1];
    __shared__ __attribute__((aligned(1024))) unsigned char first[PIECES ? 1 : G::STAGE_BYTES];
    __shared__ __attribute__((aligned(1024))) unsigned char second[PIECES ? 1 : G::STAGE_BYTES];
    unsigned char *const lds0 = PIECES ? all : first, *const lds1 = PIECES ? all + G::STAGE_BYTES : second;
    __shared__ __attribute__((aligned(1024))) unsigned char lds2[STAGES > 2 ? G::STAGE_BYTES : 1];
    __shared__ __attribute__((aligned(1024))) unsigned char lds3[STAGES > 3 ? G::STAGE_BYTES : 1];

    // This block's slice, group and tile.  The tiles of a product (of one
    // group, of all groups' rows) are walked in rasters of group_m tile rows,
    // so that blocks that run together on an XCD share operands in its L2.
    const int lane = (int)threadIdx.x & 63, xcd = (int)blockIdx.x & 7, j = (int)blockIdx.x >> 3;
    const int slots = PIECES ? p.slots : 0;
    TileSpec t;
    Piece piece;
    int tm, tn;
    auto raster = [&](int i, int rows, int &r, int &col) {
        const int per = p.group_m * p.tiles_n, first = i / per * p.group_m;
        const int high = min(rows - first, p.group_m), in = i - first * p.tiles_n;
        r = first + in % high;
        col = in / high;
    };
    if constexpr (WGRAD) {
        // every XCD takes an eighth of each group's tiles (another one from
        // group to group, for groups of few tiles): groups of many rows do not
        // pile up on one XCD
        const int tiles = p.tiles_m * p.tiles_n, per = (tiles + 7) >> 3;
        piece = xcd_piece(j, p.groups * p.splits * per, 0, slots);
        if (piece.at < 0) return;
        const int o = piece.at / per, rank = o / p.splits;
        const int i = ((xcd + o) & 7) * per + piece.at - o * per;
        if (i >= tiles) return;
        t.slice = o - rank * p.splits;
        t.group = __builtin_amdgcn_readfirstlane(group_of_rank(p.offsets, p.groups, p.rows, lane, rank));
        raster(i, p.tiles_m, tm, tn);
        group_span(p.offsets, t.group, p.rows, t.lo, t.m);
        t.lo = __builtin_amdgcn_readfirstlane(t.lo);
        t.m = __builtin_amdgcn_readfirstlane(t.m);
    } else {
        constexpr int HALF = PIECES ? BM / 2 : 0;
        const GroupRows list(p.offsets, p.groups, p.rows, BM, lane, HALF);
        // every XCD takes an eighth of either list
        auto eighth = [&](int n) { return (n + 7) >> 3; };
        auto mine = [&](int n) { return max(0, min(eighth(n), n - xcd * eighth(n))); };
        const int n = p.splits * list.total * p.tiles_n, ns = p.splits * list.small * p.tiles_n;
        piece = xcd_piece(j, mine(n), mine(ns), slots);
        if (piece.at < 0) return;
        const bool small = piece.at >= mine(n);
        const int at = small ? xcd * eighth(ns) + piece.at - mine(n) : xcd * eighth(n) + piece.at;
        const int high = small ? list.small : list.total, tiles = high * p.tiles_n;
        t.slice = at / tiles;
        raster(at - t.slice * tiles, high, tm, tn);
        list.find(p.offsets, p.groups, p.rows, BM, lane, HALF, small, tm, t.group, t.lo, t.m, tm);
    }
    t.row0 = tm * BM;
    t.col0 = tn * BN;
    if constexpr (PIECES) {
        if (piece.which >= 0) {
            t.row0 += (piece.which & 1) * (BM / 2);
            t.col0 += (piece.which >> 1 & 1) * (BN / 2);
            if (t.row0 >= (WGRAD ? p.M : t.m) || t.col0 >= p.N) return;
            // alone on their unit: three or four stages, or each k-tile waits
            // for its loads
            if (piece.which >= 4) {
                using H = Geo16<BN, BM / 2, BK, 4, 1, 3, LW, LX>;
                linear_tile<H, ALIGNED>(p, t, all, all + H::STAGE_BYTES, all + 2 * H::STAGE_BYTES, all);
                return;
            }
            using Q = Geo16<BN / 2, BM / 2, BK, 2, 2, 4, LW, LX>;
            linear_tile<Q, ALIGNED>(p, t, lds0, lds1, lds0 + Q::STAGE_BYTES, lds1 + Q::STAGE_BYTES);
            return;
        }
    }
    linear_tile<G, ALIGNED>(p, t, lds0, lds1, lds2, lds3);
}

// ---------------------------------------------------------------- few rows --

// y = act(alpha x . w + bias) + residual for groups of few rows (a decoding
// step): the weights are read once and hardly reused, so what counts is how
// many bytes of them are in flight.  A block owns 16 rows of one group and a
// strip of columns over the whole of K; its waves take turns along K, each
// streaming weights straight into registers (no LDS, no barrier in the loop,
// the next step's loads in flight under this one's products), and their sums
// meet in LDS once at the end, where the epilogue follows: one launch, no
// partial sums in memory.
//
// The products are 16 x 16 MFMAs with the 16 rows of x as one operand (rows
// past the group's last repeat it and are not stored).  Lane (q, c) = (lane /
// 16, lane % 16) supplies KV values of k (16 bytes), k = kb + KV q + i, of row
// c of x and of its column of w:
//   w as N x K: 16 bytes of row n0 + 16 f + c, one load each (W = fragments f);
//   w as K x N: KV loads of W consecutive columns n0 + W c .. of rows kb + KV q
//     + i; bf16 pairs up the rows' halves with byte permutes.  MFMA j then has
//     the columns n0 + W c + j.
// Loads use the element's alignment, whatever the pitch.
template <bool BF16, int FORM, int W, int WV>
struct FewRows {
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    static constexpr int KV = 16 / (int)sizeof(In);     // k values per lane and step
    static constexpr bool T = FORM == 1;                // w as N x K
    static constexpr int BN = 16 * W;
    static constexpr int U = T ? 4 : 8 / W;             // steps per pass
    static constexpr int KP = U * 4 * KV;               // k values per pass of a wave
    // vectors at the element's alignment
    typedef In chunk __attribute__((ext_vector_type(16 / sizeof(In)), aligned(sizeof(In))));
    typedef In piece __attribute__((ext_vector_type(W), aligned(sizeof(In))));

    static constexpr int PD = W * (int)sizeof(In) / 4;  // dwords per piece
    struct Regs {
        u32x4 x[U];
        u32x4 w[T ? U * W : 1];
        uint32_t v[T ? 1 : U * KV][T ? 1 : PD];
    };

    const In *xr;      // this lane's row of x
    const In *w;       // the group's weights
    int64_t ldw;
    int q, c, n0, N, K;

    static __device__ __forceinline__ u32x4 load_chunk(const In *p)
    {
        return __builtin_bit_cast(u32x4, *reinterpret_cast<const chunk *>(p));
    }
    // Elements e0 .. of a row, zero from `end` on.
    static __device__ __forceinline__ u32x4 load_masked(const In *row, int e0, int end)
    {
        if (e0 + KV <= end) return load_chunk(row + e0);
        union {
            u32x4 v;
            In e[KV];
        } u;
#pragma unroll
        for (int i = 0; i < KV; ++i) u.e[i] = e0 + i < end ? row[e0 + i] : In(0);
        return u.v;
    }

    // First of this lane's columns (w as K x N): the last pieces of a strip
    // that N ends in move back to end with it, and repeat columns.
    __device__ __forceinline__ int first_col() const { return min(n0 + W * c, max(N - W, 0)); }

    // One pass.  TAIL: K may end in it.  NARROW (w as K x N): N < W.
    template <bool TAIL, bool NARROW>
    __device__ __forceinline__ void load(int pass, Regs &r) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = pass * KP + (u * 4 + q) * KV;
            r.x[u] = TAIL ? load_masked(xr, k, K) : load_chunk(xr + k);
            if constexpr (T) {
#pragma unroll
                for (int f = 0; f < W; ++f) {
                    const In *row = w + (int64_t)min(n0 + 16 * f + c, N - 1) * ldw;
                    r.w[u * W + f] = TAIL ? load_masked(row, k, K) : load_chunk(row + k);
                }
            } else {
                const int col = first_col();
#pragma unroll
                for (int i = 0; i < KV; ++i) {
                    const In *row = w + (int64_t)(TAIL ? min(k + i, K - 1) : k + i) * ldw;
                    union {
                        piece v;
                        In e[W];
                        uint32_t d[PD];
                    } t;
                    if constexpr (NARROW) {
#pragma unroll
                        for (int j = 0; j < W; ++j) t.e[j] = row[min(col + j, N - 1)];
                    } else {
                        t.v = *reinterpret_cast<const piece *>(row + col);
                    }
#pragma unroll
                    for (int d = 0; d < PD; ++d) r.v[u * KV + i][d] = !TAIL || k + i < K ? t.d[d] : 0u;
                }
            }
        }
    }

    static __device__ __forceinline__ void mma(u32x4 a, u32x4 b, floatx4 &acc)
    {
        if constexpr (BF16) {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                          __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]),
                                                           acc, 0, 0, 0);
        }
    }

    __device__ __forceinline__ void compute(const Regs &r, floatx4 (&acc)[W]) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                u32x4 b;
                if constexpr (T) {
                    b = r.w[u * W + j];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (BF16)   // column j of two rows of k
                            b[i] = __builtin_amdgcn_perm(r.v[u * KV + 2 * i + 1][j / 2], r.v[u * KV + 2 * i][j / 2],
                                                         j & 1 ? 0x07060302u : 0x05040100u);
                        else
                            b[i] = r.v[u * KV + i][j];
                    }
                }
                mma(r.x[u], b, acc[j]);
            }
    }

    // This wave's passes: `wave`, `wave` + WV, ..; the last, cut one is
    // whoever's turn it is.
    template <bool NARROW>
    __device__ __forceinline__ void run(int wave, floatx4 (&acc)[W]) const
    {
        const int whole = K / KP;
        Regs cur, nxt;
        int pass = wave;
        if (pass < whole) load<false, NARROW>(pass, cur);
        for (; pass < whole; pass += WV) {
            if (pass + WV < whole) load<false, NARROW>(pass + WV, nxt);
            compute(cur, acc);
            cur = nxt;
        }
        if (pass == whole && whole * KP < K) {
            load<true, NARROW>(whole, cur);
            compute(cur, acc);
        }
    }
};

template <bool BF16, int FORM, int W, int WV>
__global__ void __launch_bounds__(64 * WV) few_rows_kernel(LinearArgs p)
{
    using F = FewRows<BF16, FORM, W, WV>;
    using In = typename F::In;
    constexpr int BM = 16, BN = F::BN;
    __shared__ float sums[WV][BM * BN];

    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const GroupRows list(p.offsets, p.groups, p.rows, BM, lane);
    // a group's row tiles next to one another: the second finds the weights in L2
    const int at = xcd_place(list.total * p.tiles_n);
    if (at < 0) return;
    const int tn = at / list.total;
    int group, lo, m, tm;
    list.find(p.offsets, p.groups, p.rows, BM, lane, 0, false, at - tn * list.total, group, lo, m, tm);
    const int row0 = lo + tm * BM, count = min(BM, m - tm * BM);

    F f;
    f.q = lane >> 4;
    f.c = lane & 15;
    f.n0 = tn * BN;
    f.N = p.N;
    f.K = p.K;
    f.ldw = p.ldw;
    f.w = static_cast<const In *>(p.w) + group * p.stride_w;
    f.xr = static_cast<const In *>(p.x) + (int64_t)(row0 + min(f.c, count - 1)) * p.ldx;

    floatx4 acc[W];
#pragma unroll
    for (int j = 0; j < W; ++j) acc[j] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (F::T || p.N >= W)
        f.template run<false>(wave, acc);
    else
        f.template run<true>(wave, acc);

    // sum r of a 16 x 16 fragment is row 4 q + r, column c
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const int col = F::T ? 16 * j + f.c : f.first_col() - f.n0 + j;
        if (F::T || col >= 0)
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[wave][(4 * f.q + r) * BN + col] = acc[j][r];
    }
    __syncthreads();
    for (int id = (int)threadIdx.x; id < count * BN; id += 64 * WV) {
        const int row = id / BN, col = f.n0 + id % BN;
        if (col >= p.N) continue;
        float v[1] = {0.0f}, bias[1];
#pragma unroll
        for (int z = 0; z < WV; ++z) v[0] += sums[z][id];
        load_bias<1>(p.e, group * p.stride_bias + col, 1, bias);
        finish_piece<1>(p.e, 0, row0 + row, col, 1, bias, v);
    }
}

}  // namespace dg
