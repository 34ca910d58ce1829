// The bf16 main loop of the linear layers, on v_mfma_f32_16x16x32_bf16.
//
// Same LDS stages, direct global->LDS loads and masked path as gemm_kernel.hpp
// (whose loaders it uses), with 16 x 16 fragments of 32 k values.  Why not the
// 32 x 32 x 16 instruction: large bf16 products run at the board's power limit,
// and there the clock follows the energy of an instruction.  Per flop the 16 x
// 16 x 32 form reads and writes half as many accumulators; registers-only loops
// of the two on random operands, back to back on one board, sustained 2059 and
// 1839 TF/s.
//
// Lane (q, c) = (lane / 16, lane % 16) holds row (or column) c and the k values
// 8 q .. 8 q + 7 of a fragment, and rows 4 q .. 4 q + 3 of column c of a sum.
#pragma once

#include "gemm_kernel.hpp"

namespace dg {

typedef float floatx4 __attribute__((ext_vector_type(4)));

// An operand tile in LDS.  k-contiguous rows are laid out as in OpTile: the 16
// lanes of a read pass take one chunk of 16 rows either way.  Outer-contiguous
// tiles are read with the LDS transpose load, 16 columns of 4 rows per 16
// lanes, and a pass of 32 lanes covers rows k .. k + 3 and k + 8 .. k + 11 of
// the same 16 columns.  The 64-byte segments of row k are permuted by k & 3, as
// in OpTile, and the 32-byte halves of each swap places in rows with bit 3
// set, so that the two groups of a pass use different banks.
template <int OUTER_, int BK_, int LAYOUT_, int NT_, int NW_>
struct OpTile16 : OpTile<true, OUTER_, BK_, LAYOUT_, NT_, NW_> {
    using Base = OpTile<true, OUTER_, BK_, LAYOUT_, NT_, NW_>;
    using Base::LAYOUT;
    static __device__ __forceinline__ int half_swap(int row) { return ((row >> 3) & 1) << 4; }
    static __device__ __forceinline__ int off(int row, int e)
    {
        return LAYOUT == KMAJOR ? Base::off(row, e) : Base::off(row, e ^ half_swap(row));
    }
    static __device__ __forceinline__ int logical(int row, int phys)
    {
        return LAYOUT == KMAJOR ? Base::logical(row, phys) : Base::logical(row, phys) ^ half_swap(row);
    }
    static __device__ __forceinline__ int logical_elem(int row, int phys)
    {
        return LAYOUT == KMAJOR ? Base::logical_elem(row, phys)
                                : Base::logical_elem(row, phys) ^ half_swap(row);
    }
};

// Tile geometry: as Geo, with 16 x 16 fragments.
template <int BM_, int BN_, int BK_, int WM_, int WN_, int STAGES_, int LA_, int LB_>
struct Geo16 {
    static constexpr bool BF16 = true;
    using In = uint16_t;
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_;
    static constexpr int STAGES = STAGES_, LA = LA_, LB = LB_;
    static constexpr int ES = 2, VEC = 8;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int FM = WTM / 16, FN = WTN / 16;   // fragments per wave
    static constexpr int STEPS = BK / 32;                // fragment steps per tile
    static_assert(BK % 32 == 0, "whole fragment steps");
    static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave sub-block: whole fragment pairs");

    using TA = OpTile16<BM, BK, LA, NT, NW>;
    using TB = OpTile16<BN, BK, LB, NT, NW>;
    static constexpr int A_BYTES = TA::BYTES;
    static constexpr int STAGE_BYTES = TA::BYTES + TB::BYTES;
    static constexpr int N_MMA = FM * FN;                // per step and wave
    static constexpr int N_DS = FM * (LA == KMAJOR ? 1 : 2) + FN * (LB == KMAJOR ? 1 : 2);
    static constexpr int LOADS_PER_TILE = (TA::PIECES + TB::PIECES) / NW;
    static constexpr int LOADS4_PER_TILE = (TA::BYTES / 256 + TB::BYTES / 256) / NW;
    static constexpr bool DMA4 =   // as Geo
        (TA::BYTES / 256) % NW == 0 && (TB::BYTES / 256) % NW == 0 &&
        (LA == MNMAJOR || TA::ROW_BYTES <= 256) && (LB == MNMAJOR || TB::ROW_BYTES <= 256) &&
        LOADS4_PER_TILE * (STAGES - 2) <= 63;
    static_assert(STAGES >= 2 && STAGES <= 4, "2 to 4 LDS stages");
    static_assert(STAGES * STAGE_BYTES <= 160 * 1024, "LDS budget of one workgroup exceeded");
    static_assert(LOADS_PER_TILE * (STAGES - 2) <= 63, "vmcnt counts at most 63 loads");
};

template <class G>
struct Frags16 {
    u32x4 a[G::FM];
    u32x4 b[G::FN];
};

// One fragment: the 8 k values from kk of outer index ob + lane % 16, kk of
// this lane's q included.
template <class T>
__device__ __forceinline__ u32x4 read_frag16(const unsigned char *tile, int lane, int ob, int kk)
{
    if constexpr (T::LAYOUT == KMAJOR) {
        return lds_load16(tile, T::off(ob + (lane & 15), kk));
    } else {
        const int s = lane & 15;
        const int col = ob + 4 * (s & 3), k = kk + (s >> 2);
        const v4i16 lo = lds_read_tr16(tile, T::off(k, col));
        const v4i16 hi = lds_read_tr16(tile, T::off(k + 4, col));
        const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
        return u32x4{l[0], l[1], h[0], h[1]};
    }
}

template <class G>
__device__ __forceinline__ void load_frags16(const unsigned char *stage, const BlockCtx<G> &c, int step,
                                             Frags16<G> &f)
{
    const int kk = step * 32 + 8 * (c.lane >> 4);
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
        f.a[i] = read_frag16<typename G::TA>(stage, c.lane, c.wrow * G::WTM + i * 16, kk);
#pragma unroll
    for (int j = 0; j < G::FN; ++j)
        f.b[j] = read_frag16<typename G::TB>(stage + G::A_BYTES, c.lane, c.wcol * G::WTN + j * 16, kk);
}

template <class G>
__device__ __forceinline__ void mma16(const Frags16<G> &f, floatx4 (&acc)[G::FM][G::FN])
{
#pragma unroll
    for (int i = 0; i < G::FM; ++i)
#pragma unroll
        for (int j = 0; j < G::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.a[i]),
                                                                __builtin_bit_cast(bf16x8, f.b[j]),
                                                                acc[i][j], 0, 0, 0);
}

// Two MFMAs, then up to one direct load and one LDS read, and so on: as
// interleave_step, for MFMAs of half the length.
template <int N_MMA, int N_DS, int N_VMEM>
__device__ __forceinline__ void interleave16()
{
#pragma unroll
    for (int i = 0; i < N_MMA / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);                  // MFMA
        if (i < N_VMEM) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
        if (i < N_DS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // DS read
    }
    if (N_DS > N_MMA / 2) __builtin_amdgcn_sched_group_barrier(0x100, N_DS - N_MMA / 2, 0);
    if (N_VMEM > N_MMA / 2) __builtin_amdgcn_sched_group_barrier(0x020, N_VMEM - N_MMA / 2, 0);
}

// One k-tile: the steps of the tile in `stage`, while the tile at k_load
// streams into `load`; after the wait for the next tile and the barrier its
// first fragments are read under the last step's products.
template <class G, int DW>
__device__ __forceinline__ void direct_tile16(const unsigned char *stage, const unsigned char *next,
                                              unsigned char *load, const BlockCtx<G> &c,
                                              const DirectOffsets<G, DW> &o, int k_load, Frags16<G> &cur,
                                              floatx4 (&acc)[G::FM][G::FN])
{
    constexpr int LOADS = DirectOffsets<G, DW>::LOADS_PER_TILE;
    Frags16<G> nxt;
    direct_tile_load(load, c, o, k_load);
#pragma unroll
    for (int step = 0; step < G::STEPS - 1; ++step) {
        load_frags16(stage, c, step + 1, nxt);
        mma16(cur, acc);
        interleave16<G::N_MMA, G::N_DS, 0>();
        cur = nxt;
    }
    // lgkmcnt(0): this tile's reads are done before anyone may overwrite it
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(LOADS * (G::STAGES - 2)));
    __builtin_amdgcn_s_barrier();
    load_frags16(next, c, 0, nxt);
    mma16(cur, acc);
    interleave16<G::N_MMA, G::N_DS, 0>();
    cur = nxt;
}

// Whole k-tiles [0, ntiles) from k_first, in the order c.rot, c.rot + 1, .. of
// the tiles taken round, as main_loop_direct: distinct restrict stages, STAGES
// tiles per iteration, loads past the last tile wrap round to tiles already
// done.  On entry no wave may read or load any stage;
// on exit no load is in flight.
template <class G, int DW>
__device__ __forceinline__ void main_loop16_direct(unsigned char *__restrict__ s0,
                                                   unsigned char *__restrict__ s1,
                                                   unsigned char *__restrict__ s2,
                                                   unsigned char *__restrict__ s3, const BlockCtx<G> &c,
                                                   int k_first, int ntiles, floatx4 (&acc)[G::FM][G::FN])
{
    constexpr int S = G::STAGES, BK = G::BK;
    constexpr int LOADS = DirectOffsets<G, DW>::LOADS_PER_TILE;
    static_assert(LOADS * (S - 2) <= 63, "vmcnt counts at most 63 loads");
    unsigned char *const st[4] = {s0, s1, s2, s3};
    Frags16<G> cur;
    DirectOffsets<G, DW> o;
    tile_offsets(c.tid >> 6, c.lane, c.lda, c.bm, c.M, o.a);
    tile_offsets(c.tid >> 6, c.lane, c.ldb, c.bn, c.N, o.b);
    int kt = c.rot % ntiles;
    auto next_k = [&]() {
        const int k = k_first + kt * BK;
        kt = kt + 1 == ntiles ? 0 : kt + 1;
        return k;
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) direct_tile_load(st[s], c, o, next_k());
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(LOADS * (S - 2)));
    __builtin_amdgcn_s_barrier();
    load_frags16(st[0], c, 0, cur);
    for (int t = 0; t < ntiles; t += S) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s == 0 || t + s < ntiles)
                direct_tile16(st[s], st[(s + 1) % S], st[(s + S - 1) % S], c, o, next_k(), cur, acc);
        }
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __builtin_amdgcn_s_barrier();
}

// `ntiles` masked k-tiles from k_first through registers, as main_loop_masked.
template <class G, class Loader>
__device__ __forceinline__ void main_loop16_masked(unsigned char *smem0, unsigned char *smem1,
                                                   const BlockCtx<G> &c, int k_first, int ntiles,
                                                   floatx4 (&acc)[G::FM][G::FN], Loader &&load)
{
    StageRegs<G> regs;
    Frags16<G> f;
    load(k_first, regs);
    lds_store(smem0, c.tid, regs);
    __syncthreads();
    for (int t = 0; t < ntiles; ++t) {
        unsigned char *stage = (t & 1) ? smem1 : smem0;
        unsigned char *other = (t & 1) ? smem0 : smem1;
        const bool more = t + 1 < ntiles;
        if (more) load(k_first + (t + 1) * G::BK, regs);
#pragma unroll
        for (int step = 0; step < G::STEPS; ++step) {
            load_frags16(stage, c, step, f);
            mma16(f, acc);
        }
        if (more) lds_store(other, c.tid, regs);
        __syncthreads();
    }
}

// ------------------------------------------------------------ pinned order ---

// Nothing moves across.
__device__ __forceinline__ void slot_fence()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void slot_end()
{
    slot_fence();
    __builtin_amdgcn_s_barrier();
    slot_fence();
}

// The loop for blocks with one wave per SIMD and large wave tiles: the order of
// products, LDS reads and direct loads is written out and pinned, since no
// second wave fills a gap.
//
// Why large wave tiles: a wave reads FM + FN fragments of LDS for FM FN
// products.  At 128 x 64 per wave (eight waves on 256 x 256) the reads and the
// loads' writes of a k-tile take the LDS as long as its products take the
// matrix cores; at 128 x 128 (four waves), three quarters.
//
// Two k-steps of 32 per tile.  During step 0 of tile t the fragments of step 1
// are read; then the stage of tile t is consumed.  The tile's one barrier stands
// here: every wave has waited for its reads of tile t and for its direct loads
// of tile t + 1, so afterwards the loads of tile t + 2 may overwrite the stage
// and the first fragments of tile t + 1 may be read, both during step 1.  The
// loads are spread over all of step 1 (in its first half they came faster than
// the LDS takes them, and stood before the products: bf16 zeros, 4096 x 4096 x
// 8192, 157 against 136 us) and waited for at the end of the next step 0.
//
// The products go in 2 x 2 blocks of fragments, each product sharing an operand
// with the one before: 1.7% over rows of fragments at the board's power limit.
template <class G>
struct PinnedLoop {
    static constexpr bool OK = G::STEPS == 2 && G::STAGES == 2 && G::FM % 2 == 0 && G::FN % 2 == 0;
    static constexpr int GROUPS = G::N_MMA / 4;        // of four products
    static constexpr int FRAGS = G::FM + G::FN;

    // The n-th fragment in the order that the products of a step need them:
    // the B fragments and the first A fragment, then the other A fragments.
    template <int N>
    static __device__ __forceinline__ void read(const unsigned char *stage, const BlockCtx<G> &c, int step,
                                                Frags16<G> &f)
    {
        const int kk = step * 32 + 8 * (c.lane >> 4);
        if constexpr (N == 0)
            f.a[0] = read_frag16<typename G::TA>(stage, c.lane, c.wrow * G::WTM, kk);
        else if constexpr (N <= G::FN)
            f.b[N - 1] = read_frag16<typename G::TB>(stage + G::A_BYTES, c.lane,
                                                     c.wcol * G::WTN + (N - 1) * 16, kk);
        else
            f.a[N - G::FN] = read_frag16<typename G::TA>(stage, c.lane,
                                                         c.wrow * G::WTM + (N - G::FN) * 16, kk);
    }

    // One step: the products of `f`, with the fragments of `step` of `from`
    // read into `next` and `loads(i)`, i < NL, issued between them: the reads in
    // the first three quarters of the groups, the loads in all.
    template <int NL, class Load>
    static __device__ __forceinline__ void step(const Frags16<G> &f, const unsigned char *from,
                                                const BlockCtx<G> &c, int s, Frags16<G> &next,
                                                floatx4 (&acc)[G::FM][G::FN], Load &&loads)
    {
        constexpr int GR = GROUPS * 3 / 4 > 0 ? GROUPS * 3 / 4 : 1;
        static_for<0, GROUPS>([&](auto g_c) {
            constexpr int g = decltype(g_c)::value;
            static_for<NL * g / GROUPS, NL *(g + 1) / GROUPS>([&](auto i) { loads(i); });
            if constexpr (g < GR)
                static_for<FRAGS * g / GR, FRAGS *(g + 1) / GR>(
                    [&](auto n) { read<decltype(n)::value>(from, c, s, next); });
            // block g: (0, 0) (0, 1) (1, 1) (1, 0) of fragments 2 x 2
            static_for<0, 4>([&](auto m_c) {
                constexpr int m = decltype(m_c)::value;
                constexpr int i = g / (G::FN / 2) * 2 + m / 2;
                constexpr int j = g % (G::FN / 2) * 2 + (m == 1 || m == 2 ? 1 : 0);
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.a[i]),
                                                                    __builtin_bit_cast(bf16x8, f.b[j]),
                                                                    acc[i][j], 0, 0, 0);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    }
};

// Whole k-tiles [0, ntiles), ntiles > 0, from k_first, through 16-byte direct
// loads, in the order c.rot, c.rot + 1, .. of the tiles taken round.  On entry
// no wave may read or load any stage; on exit no load is in flight and all
// waves have passed a barrier after their last read.
template <class G>
__device__ __forceinline__ void main_loop_pinned(unsigned char *s0, unsigned char *s1, const BlockCtx<G> &c,
                                                 int k_first, int ntiles, floatx4 (&acc)[G::FM][G::FN])
{
    using L = PinnedLoop<G>;
    using TA = typename G::TA;
    using TB = typename G::TB;
    static_assert(L::OK, "two steps and two stages");
    constexpr int PA = TileOffsets<TA, 16>::PER_WAVE, PB = TileOffsets<TB, 16>::PER_WAVE;
    unsigned char *const st[2] = {s0, s1};
    DirectOffsets<G, 16> o;
    tile_offsets(c.tid >> 6, c.lane, c.lda, c.bm, c.M, o.a);
    tile_offsets(c.tid >> 6, c.lane, c.ldb, c.bn, c.N, o.b);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(c.tid >> 6);
    // the t-th tile visited, from tile c.rot on; past the last one the loads
    // repeat it: in bounds, and never read
    const int rot = c.rot % ntiles;
    auto k_of = [&](int t) {
        const int u = min(t, ntiles - 1) + rot;
        return k_first + (u >= ntiles ? u - ntiles : u) * G::BK;
    };
    Frags16<G> f0, f1;

    direct_tile_load(st[0], c, o, k_of(0));
    direct_tile_load(st[1], c, o, k_of(1));
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(PA + PB));
    slot_end();
    static_for<0, L::FRAGS>([&](auto n) { L::template read<decltype(n)::value>(st[0], c, 0, f0); });
    slot_fence();
    for (int t0 = 0; t0 < ntiles; t0 += 2) {
        static_for<0, 2>([&](auto s_c) {
            constexpr int s = decltype(s_c)::value;
            const int t = t0 + s;
            if (s > 0 && t >= ntiles) return;
            L::template step<0>(f0, st[s], c, 1, f1, acc, [](auto) {});
            __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
            slot_end();
            const int k = k_of(t + 2);
            const unsigned char *a_base =
                reinterpret_cast<const unsigned char *>(c.A) + tile_origin_bytes<TA>(c.lda, c.bm, k);
            const unsigned char *b_base =
                reinterpret_cast<const unsigned char *>(c.B) + tile_origin_bytes<TB>(c.ldb, c.bn, k);
            const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(st[s])) + 1024 * wave;
            L::template step<PA + PB>(f1, st[1 - s], c, 0, f0, acc, [&](auto i_c) {
                constexpr int i = decltype(i_c)::value;
                if constexpr (i < PA)
                    direct_load16(a_base, o.a.v[i], lds + 1024 * G::NW * i);
                else
                    direct_load16(b_base, o.b.v[i - PA], lds + G::A_BYTES + 1024 * G::NW * (i - PA));
            });
        });
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    slot_end();
}

}  // namespace dg
