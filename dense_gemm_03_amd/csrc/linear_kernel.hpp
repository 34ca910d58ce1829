// Device code of the linear layers: the tiled product of gemm_kernel.hpp with
// row groups and an epilogue of its own.
//
//     y = act(alpha x . w + bias) + beta_c residual        (LA == KMAJOR)
//     dw = alpha x^T . dz + beta dw                        (LA == MNMAJOR)
//
// In the first form the groups cut the rows of the output: a group's rows are
// covered by tiles of BM rows of their own, so a tile never mixes two weight
// matrices, and the tile list is worked out on the device from the offsets
// (GroupRows).  In the second the groups cut the summed axis: every group has
// an output matrix, and its blocks walk that group's rows only.
#pragma once

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
    const void *A, *B;      // x and w, or x^T and dz (or dz^T and x)
    const int32_t *offsets; // nullptr: one group of all rows
    float *ws;              // partial sums of `splits` > 1 slices
    EpilogueArgs e;
    int64_t lda, ldb;
    int64_t stride_b;       // elements between the groups' w (first form)
    int64_t stride_c;       // elements between the groups' dw (second form)
    int64_t stride_bias;
    int rows;               // rows of x: M of the first form, K of the second
    int M, N, K;            // extents of one group's product; the first form's M and the
                            // second's K are replaced by the group's row count
    int m_load, n_load;     // as KernelArgs
    int groups;             // at least 1
    int tiles_m, tiles_n;   // tiles_m: second form only
    int splits, k_per_split;
    int group_m;
    int direct_ok;
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

// act(z) of V values, the activation chosen once for all of them.
template <int V>
__device__ __forceinline__ void act_apply(int act, float (&v)[V])
{
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] <= 0.0f ? 0.0f : v[i];   // a NaN stays
        break;
    case ACT_GELU:
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.5f * v[i] * (1.0f + erff(0.70710678118654752f * v[i]));
        break;
    case ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid(v[i] * (kGeluA + kGeluB * v[i] * v[i]));
        break;
    case ACT_SILU:
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid(v[i]);
        break;
    default: break;
    }
}

// act'(z), written over z.  Beyond |z| = 100 every slope here is 0 or 1 to
// more digits than fp32 holds; the bound keeps its products of a vanishing
// and a growing factor from forming 0 x infinity.  A NaN stays.
template <int V>
__device__ __forceinline__ void act_slope(int act, float (&v)[V])
{
    auto bounded = [](float z) { return z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z; };
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] > 0.0f ? 1.0f : v[i] <= 0.0f ? 0.0f : v[i];
        break;
    case ACT_GELU:   // Phi(z) + z phi(z)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = bounded(v[i]);
            v[i] = 0.5f * (1.0f + erff(0.70710678118654752f * z)) +
                   z * 0.39894228040143268f * __builtin_amdgcn_exp2f(-0.72134752f * z * z);
        }
        break;
    case ACT_GELU_TANH:   // q + z q (1 - q) u',  q = sigmoid(u)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = bounded(v[i]);
            const float q = sigmoid(z * (kGeluA + kGeluB * z * z));
            v[i] = q + z * q * (1.0f - q) * (kGeluA + 3.0f * kGeluB * z * z);
        }
        break;
    case ACT_SILU:   // q (1 + z (1 - q)),  q = sigmoid(z)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float z = bounded(v[i]);
            const float q = sigmoid(z);
            v[i] = q * (1.0f + z * (1.0f - q));
        }
        break;
    default:
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 1.0f;
        break;
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
// the lanes), so no launch before this one and no memory is needed.
struct GroupRows {
    int total;   // tiles of all groups

    __device__ __forceinline__ static int lane_tiles(const int32_t *offsets, int g, int groups,
                                                     int rows, int bm, int &lo, int &m)
    {
        lo = 0;
        m = 0;
        if (g < groups) group_span(offsets, g, rows, lo, m);
        return (m + bm - 1) / bm;
    }
    __device__ __forceinline__ static int scan(int v, int lane)
    {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(v, d);
            if (lane >= d) v += o;
        }
        return v;
    }
    __device__ __forceinline__ GroupRows(const int32_t *offsets, int groups, int rows, int bm, int lane)
    {
        total = 0;
        if (offsets == nullptr) {
            total = (rows + bm - 1) / bm;
            return;
        }
        for (int base = 0; base < groups; base += 64) {
            int lo, m;
            const int t = scan(lane_tiles(offsets, base + lane, groups, rows, bm, lo, m), lane);
            total += __builtin_amdgcn_readlane(t, 63);
        }
    }
    // Group, its first row, its rows and the tile inside it of tile `t` < total.
    __device__ __forceinline__ void find(const int32_t *offsets, int groups, int rows, int bm,
                                         int lane, int t, int &group, int &lo, int &m, int &tm) const
    {
        group = 0;
        lo = 0;
        m = rows;
        tm = t;
        if (offsets == nullptr) return;
        int before = 0;
        for (int base = 0; base < groups; base += 64) {
            int l, n;
            const int mine = lane_tiles(offsets, base + lane, groups, rows, bm, l, n);
            const int upto = before + scan(mine, lane);
            const uint64_t past = __ballot(upto > t);
            if (past != 0) {
                const int at = __builtin_ctzll(past);
                group = base + at;
                lo = __builtin_amdgcn_readlane(l, at);
                m = __builtin_amdgcn_readlane(n, at);
                tm = t - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(mine, at));
                return;
            }
            before = __builtin_amdgcn_readlane(upto, 63);
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

// --------------------------------------------------------------- epilogue --

template <int V>
__device__ __forceinline__ void load_out(const void *C, int64_t idx, int n, bool bf16, bool vec,
                                         float (&v)[V])
{
    if (bf16) {
        const uint16_t *c = static_cast<const uint16_t *>(C) + idx;
        if (V == 8 && vec && n >= V) {
            const u32x4 w = load16(c);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                v[2 * i] = __uint_as_float(w[i & 3] << 16);
                v[2 * i + 1] = __uint_as_float(w[i & 3] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = i < n ? __uint_as_float((uint32_t)c[i] << 16) : 0.0f;
        }
    } else {
        const float *c = static_cast<const float *>(C) + idx;
        if (V == 4 && vec && n >= V) {
            const u32x4 w = load16(c);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i & 3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = i < n ? c[i] : 0.0f;
        }
    }
}

// Rounded once, to nearest even (bf16), or as they are.  Non-temporal: the
// layer's outputs are written once and must not evict the operand tiles that
// other blocks still stream.
template <int V>
__device__ __forceinline__ void store_outs(void *C, int64_t idx, int n, bool bf16, bool vec,
                                           const float (&v)[V])
{
    if (bf16) {
        uint16_t *c = static_cast<uint16_t *>(C) + idx;
        if (V == 8 && vec && n >= V) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i & 3] = f32x2_to_bf16x2_rne(v[2 * i], v[2 * i + 1]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(c));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) c[i] = f32_to_bf16_rne(v[i]);
        }
    } else {
        float *c = static_cast<float *>(C) + idx;
        if (V == 4 && vec && n >= V) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < V; ++i) w[i & 3] = __float_as_uint(v[i]);
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(c));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) c[i] = v[i];
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
template <int V>
__device__ __forceinline__ void finish_piece(const EpilogueArgs &e, int64_t c_off, int64_t row,
                                             int col, int n, const float (&bias)[V], float (&v)[V])
{
    const bool bf16 = e.out_bf16 != 0, vec = e.vec != 0;
    float old[V];
    if (e.residual != nullptr) load_out<V>(e.residual, c_off + row * e.ldr + col, n, bf16, vec, old);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e.alpha * v[i] + bias[i];
    if (e.pre != nullptr) store_outs<V>(e.pre, row * e.ldp + col, n, bf16, vec, v);
    act_apply<V>(e.act, v);
    if (e.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += e.beta * old[i];
    }
    store_outs<V>(e.C, c_off + row * e.ldc + col, n, bf16, vec, v);
}

// The block's accumulators, finished and stored (or stored raw, as partial
// sums).  A fragment gives each lane single elements of 32 columns, so each
// wave passes one 32-row fragment row at a time through LDS (its own scratch
// in the stages, free after the main loop) and takes it back as pieces of V
// consecutive columns -- 16 bytes of output -- per lane.  64 lanes cover whole
// rows of the wave's sub-block, so a lane's column is the same in every piece
// and its bias is loaded once.  Blocks at an edge and rows without 16-byte
// alignment go the same way with masked element accesses.
template <class G, int V>
struct FinishTile {
    static constexpr int CPR = G::WTN / V;        // pieces per row
    static constexpr int RPI = 64 / CPR;          // rows per pass of the wave
    static constexpr int SCRATCH = 32 * G::WTN * 4;
    static constexpr int PER_STAGE = G::STAGE_BYTES / SCRATCH;
    static_assert(PER_STAGE * G::STAGES >= G::NW, "one scratch per wave");
    static_assert(64 % CPR == 0 && 32 % RPI == 0, "whole rows per pass");
    // Columns move in groups so that the lanes of a fragment write use other
    // banks: 32 x 32 fragments (fp32) write rows 4 apart in two lane halves,
    // 16 x 16 ones (bf16) in four quarters.
    static __device__ __forceinline__ int place(int row, int col)
    {
        if (G::BF16) return col ^ (((row >> 2) & (G::WTN >= 64 ? 3 : 1)) << 4);
        return G::WTN >= 64 ? col ^ (((row >> 2) & 1) << 5) : col;
    }
    static __device__ __forceinline__ void put(unsigned char *scr, int row, int col, float v)
    {
        *reinterpret_cast<float *>(scr + 4 * (row * G::WTN + place(row, col))) = v;
    }

    template <class Acc, class Out>
    static __device__ __forceinline__ void run(unsigned char *scr, const BlockCtx<G> &c, const Acc &acc,
                                               Out &&out)
    {
        const int cc = V * (c.lane % CPR), r0 = c.lane / CPR;
        static_for<0, G::WTM / 32>([&](auto fm) {
            if constexpr (G::BF16) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int fn = 0; fn < G::FN; ++fn)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            put(scr, 16 * h + 4 * (c.lane >> 4) + r, fn * 16 + (c.lane & 15),
                                acc[2 * fm + h][fn][r]);
            } else {
#pragma unroll
                for (int fn = 0; fn < G::FN; ++fn)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        put(scr, 8 * (r >> 2) + 4 * (c.lane >> 5) + (r & 3), fn * 32 + (c.lane & 31),
                            acc[fm][fn][r]);
            }
            // a wave's LDS accesses complete in order: the reads see the
            // writes above, and the next rows' writes follow these reads
#pragma unroll 2
            for (int u = 0; u < 32 / RPI; ++u) {
                const int rr = r0 + u * RPI;
                float v[V];
#pragma unroll
                for (int h = 0; h < V; h += 4) {
                    const u32x4 w = lds_load16(scr, 4 * (rr * G::WTN + place(rr, cc + h)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[h + i] = __uint_as_float(w[i]);
                }
                out(c.wrow * G::WTM + fm * 32 + rr, v);
            }
        });
    }
};

// ------------------------------------------------------------------ kernel --

template <bool BF16, int BM, int BN, int BK, int WM, int WN, int STAGES, int LA, int LB, bool ALIGNED>
__global__ void __launch_bounds__(64 * WM * WN) linear_kernel(LinearArgs p)
{
    using G = typename std::conditional<BF16, Geo16<BM, BN, BK, WM, WN, STAGES, LA, LB>,
                                        Geo<BF16, BM, BN, BK, WM, WN, STAGES, LA, LB>>::type;
    using In = typename G::In;
    using Sum = typename std::conditional<BF16, floatx4, floatx16>::type;
    constexpr int SUMS = BF16 ? 4 : 16;
    constexpr bool PINNED = BF16 && WM * WN == 4 && BK == 64 && STAGES == 2 && ALIGNED;
    constexpr bool TWO = BF16 && WM * WN == 8 && STAGES == two_groups_stages(BM / WM / 16);
    constexpr bool WGRAD = LA == MNMAJOR;   // groups cut the summed axis

    __shared__ __attribute__((aligned(1024))) unsigned char lds0[G::STAGE_BYTES];
    __shared__ __attribute__((aligned(1024))) unsigned char lds1[G::STAGE_BYTES];
    __shared__ __attribute__((aligned(1024))) unsigned char lds2[STAGES > 2 ? G::STAGE_BYTES : 1];
    __shared__ __attribute__((aligned(1024))) unsigned char lds3[STAGES > 3 ? G::STAGE_BYTES : 1];

    BlockCtx<G> c;
    c.tid = (int)threadIdx.x;
    c.lane = c.tid & 63;
    const int wave = c.tid >> 6;
    c.wrow = wave / WN;
    c.wcol = wave % WN;

    // This block's slice, group and tile.
    int slice, group, lo, m, tm, tn;
    if constexpr (WGRAD) {
        const int tiles = p.tiles_m * p.tiles_n;
        const int at = xcd_place(p.splits * p.groups * tiles);
        if (at < 0) return;
        slice = at / (p.groups * tiles);
        const int rest = at - slice * p.groups * tiles;
        group = rest / tiles;
        const int t = rest - group * tiles;
        const int per_raster = p.group_m * p.tiles_n;
        const int first = t / per_raster * p.group_m;
        const int rows = min(p.tiles_m - first, p.group_m);
        const int in = t - first * p.tiles_n;
        tm = first + in % rows;
        tn = in / rows;
        group_span(p.offsets, group, p.rows, lo, m);
        lo = __builtin_amdgcn_readfirstlane(lo);
        m = __builtin_amdgcn_readfirstlane(m);
    } else {
        const GroupRows list(p.offsets, p.groups, p.rows, BM, c.lane);
        const int tiles = list.total * p.tiles_n;
        const int at = xcd_place(p.splits * tiles);
        if (at < 0) return;
        slice = at / tiles;
        const int t = at - slice * tiles;
        const int per_raster = p.group_m * p.tiles_n;
        const int first = t / per_raster * p.group_m;
        const int rows = min(list.total - first, p.group_m);
        const int in = t - first * p.tiles_n;
        tn = in / rows;
        list.find(p.offsets, p.groups, p.rows, BM, c.lane, first + in % rows, group, lo, m, tm);
    }
    c.bm = tm * BM;
    c.bn = tn * BN;
    c.lda = p.lda;
    c.ldb = p.ldb;
    c.A = static_cast<const In *>(p.A) + (int64_t)lo * p.lda;
    c.N = p.n_load;
    int K, kps;
    if constexpr (WGRAD) {
        c.B = static_cast<const In *>(p.B) + (int64_t)lo * p.ldb;
        c.M = p.m_load;
        K = m;
        // whole k-tiles per slice; a slice past the group's rows sums nothing
        kps = ((m + BK - 1) / BK + p.splits - 1) / p.splits * BK;
    } else {
        c.B = static_cast<const In *>(p.B) + group * p.stride_b;
        c.M = m;
        K = p.K;
        kps = p.k_per_split;
    }
    const int kbeg = min(K, slice * kps);
    c.kend = min(K, kbeg + kps);
    const int ntiles = (c.kend - kbeg + BK - 1) / BK;

    Sum acc[G::FM][G::FN];
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < G::FN; ++fn)
#pragma unroll
            for (int r = 0; r < SUMS; ++r) acc[fm][fn][r] = 0.0f;
    auto direct = [&](auto dw, int nfast, int kbeg) {
        constexpr int DW = decltype(dw)::value;
        if constexpr (BF16 && PINNED) {
            static_assert(DW == 16, "aligned rows");
            main_loop_pinned<G>(lds0, lds1, c, kbeg, nfast, acc);
        } else if constexpr (BF16 && TWO) {
            const bool busy = c.bm + c.wrow * G::WTM < c.M && c.bn + c.wcol * G::WTN < c.N;
            main_loop_two_groups<G, DW>(lds0, lds1, lds2, c, kbeg, nfast,
                                        __builtin_amdgcn_readfirstlane(busy), acc);
        } else if constexpr (BF16)
            main_loop16_direct<G, DW>(lds0, lds1, lds2, lds3, c, kbeg, nfast, acc);
        else
            main_loop_direct<G, decltype(dw)::value>(lds0, lds1, lds2, lds3, c, kbeg, nfast, acc);
    };

    // The main loops and the choice between them are those of the dense
    // product, on the group's rows: whole k-tiles through direct loads of 16
    // bytes per lane (aligned rows) or 4 range-checked ones, the rest masked.
    {
        const bool edge_mn = c.bm + BM > c.M || c.bn + BN > c.N;
        const bool edge16 = (G::LA == KMAJOR || c.M % G::VEC == 0) &&
                            (G::LB == KMAJOR || c.N % G::VEC == 0);
        const bool x4 = ALIGNED && p.direct_ok && (!edge_mn || edge16);
        const bool pairs_ok =
            !G::BF16 || (((p.lda | p.ldb) & 1) == 0 && (((uintptr_t)c.A | (uintptr_t)c.B) & 3) == 0 &&
                         (G::LA == KMAJOR || (c.M & 1) == 0) && (G::LB == KMAJOR || (c.N & 1) == 0));
        const bool dw = G::DMA4 && !PINNED && p.direct_ok && pairs_ok && !x4;
        const int nfast = x4 || dw ? (c.kend - kbeg) / BK : 0;
        c.rot = (tm + tn) % 8;
        if constexpr (G::DMA4 && !PINNED) {
            c.a_end = operand_end_bytes<typename G::TA>(p.lda, c.M, K);
            c.b_end = operand_end_bytes<typename G::TB>(p.ldb, c.N, K);
            if (dw && nfast > 0) direct(std::integral_constant<int, 4>(), nfast, kbeg);
        }
        if constexpr (ALIGNED) {
            if (x4 && nfast > 0) direct(std::integral_constant<int, 16>(), nfast, kbeg);
        }
        if (ntiles > nfast) {
            auto load = [&](int k0, StageRegs<G> &r) { global_load_masked<ALIGNED>(c, k0, r); };
            if constexpr (BF16)
                main_loop16_masked(lds0, lds1, c, kbeg + nfast * BK, ntiles - nfast, acc, load);
            else
                main_loop_masked(lds0, lds1, c, kbeg + nfast * BK, ntiles - nfast, acc, load);
        }
    }

    // Epilogue.  The waves' scratches share the stages: wait until the last
    // reader of them is done.
    __syncthreads();
    using F = FinishTile<G, 4>;
    const int wv = __builtin_amdgcn_readfirstlane(wave);
    const int arr = wv / F::PER_STAGE;
    unsigned char *scr = (arr == 0 ? lds0 : arr == 1 ? lds1 : arr == 2 ? lds2 : lds3) +
                         (wv % F::PER_STAGE) * F::SCRATCH;
    const int out_rows = WGRAD ? p.M : m;   // rows of this group's output
    if (p.splits > 1) {
        // raw sums, summed by the reduce kernel: slice-major, first form rows x
        // N by global row, second form groups x M x N
        const int64_t row0 = WGRAD ? ((int64_t)slice * p.groups + group) * p.M
                                   : (int64_t)slice * p.rows + lo;
        const int col = c.bn + c.wcol * G::WTN + 4 * (c.lane % F::CPR);
        F::run(scr, c, acc, [&](int r, float (&v)[4]) {
            const int row = c.bm + r;
            if (row >= out_rows) return;
            float *out = p.ws + (row0 + row) * p.N + col;
            if ((p.N & 3) == 0) {
                if (col < p.N) *reinterpret_cast<u32x4 *>(out) = __builtin_bit_cast(u32x4, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < p.N) out[i] = v[i];
            }
        });
        return;
    }
    const int64_t crow0 = WGRAD ? 0 : lo;
    const int64_t c_off = WGRAD ? group * p.stride_c : 0;
    auto finish = [&](auto v_c) {
        constexpr int V = decltype(v_c)::value;
        using FV = FinishTile<G, V>;
        const int col = c.bn + c.wcol * G::WTN + V * (c.lane % FV::CPR);
        const int n = p.N - col;
        float bias[V];
        load_bias<V>(p.e, group * p.stride_bias + col, n, bias);
        FV::run(scr, c, acc, [&](int r, float (&v)[V]) {
            const int row = c.bm + r;
            if (row < out_rows && n > 0) finish_piece<V>(p.e, c_off, crow0 + row, col, n, bias, v);
        });
    };
    if (p.e.out_bf16)
        finish(std::integral_constant<int, 8>());
    else
        finish(std::integral_constant<int, 4>());
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
    list.find(p.offsets, p.groups, p.rows, BM, lane, at - tn * list.total, group, lo, m, tm);
    const int row0 = lo + tm * BM, count = min(BM, m - tm * BM);

    F f;
    f.q = lane >> 4;
    f.c = lane & 15;
    f.n0 = tn * BN;
    f.N = p.N;
    f.K = p.K;
    f.ldw = p.ldb;
    f.w = static_cast<const In *>(p.B) + group * p.stride_b;
    f.xr = static_cast<const In *>(p.A) + (int64_t)(row0 + min(f.c, count - 1)) * p.lda;

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
