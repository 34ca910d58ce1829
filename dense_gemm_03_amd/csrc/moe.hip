// A whole mixture-of-experts layer for a few tokens, in two kernels:
//
//     h[t, j] = act(x_t . gate_e) * (x_t . up_e)   (or act(x_t . up_e)),   e = ids[t, j]
//     y_t = sum_j weights[t, j] h[t, j] . down_e + residual_t
//
// Bound by HBM: the weights of the experts that have a token are read once, the
// rest is small.  So what counts is how many bytes of weights are in flight: waves
// stream them straight into registers (no LDS, no barrier in the loops, the next
// step's loads under way during this one's products), and every block works out
// for itself which experts have tokens, and which, from the ids: no launch sorts
// them, and no weights are read for an expert without tokens.
//
// Up to 16 tokens, an expert's tokens are one tile of rows of 16 x 16 MFMAs, and a
// block of the second product goes through all experts for a strip of y, which it
// finishes.  Beyond, blocks of both products take one expert each, up to 64 rows at a
// time (its weights are read once per 64 tokens that name it), and a third kernel adds
// up the experts' rows of a token.  A token that names an expert twice is one row with
// both its weights.
//
// Times of a call among others, bf16: 1 token to 4 of 32 experts of 4096 x 2048, N x K
// weights (201 MB) 44 us, 4.5 TB/s; 16 tokens to 8 of 64 of 2048 x 1024 each, K x N (698 MB
// of the experts that they name) 134 us, 5.2 TB/s; 64 tokens over 8 of 4096 x 8192, N x K
// (1.6 GB) 321 to 339 us, 4.8 to 5.0 TB/s.  A 4 GiB copy moves 4.8 to 5.4 TB/s.
#include "serving.hpp"
#include "strip.hpp"

namespace dg {
namespace {

// ------------------------------------------------------- experts and tokens --

constexpr int MAX_EXPERTS = MOE_MAX_EXPERTS;

// Marks the experts that the ids name, by the block; ids out of range name none.
template <int WV>
__device__ __forceinline__ void mark_experts(const int32_t *ids, int count, int experts, uint32_t *bits, int tid)
{
    const int32_t first = tid < count ? ids[tid] : -1;   // under way while the bits are cleared
    if (tid < MAX_EXPERTS / 32) bits[tid] = 0;
    __syncthreads();
    for (int i = tid; i < count; i += 64 * WV) {
        const int32_t id = i == tid ? first : ids[i];
        if ((unsigned)id < (unsigned)experts) atomicOr(&bits[(unsigned)id >> 5], 1u << (id & 31));
    }
    __syncthreads();
}

// This block's place in a list of `count`.  Strips of w as K x N that lie side by side
// share cache lines: they run on one XCD (16 tokens, 64 experts of 2048 x 1024: 163 us,
// spread 168).  Strips of w as N x K share nothing, and spread (64 tokens, 8 experts of
// 4096 x 8192: 440 us, side by side on one XCD 520).
template <bool T>
__device__ __forceinline__ int place_of_block(int count)
{
    if constexpr (!T) return xcd_place(count);
    return (int)blockIdx.x < count ? (int)blockIdx.x : -1;
}

// Sum over the lanes below and this one.
__device__ __forceinline__ int scan(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// The u-th expert of the set, or -1.
__device__ __forceinline__ int expert_at(const uint32_t *bits, int u, int lane)
{
    uint32_t w = lane < MAX_EXPERTS / 32 ? bits[lane] : 0;
    const int own = __builtin_popcount(w), upto = scan(own, lane);
    const uint64_t past = __ballot(upto > u);
    if (past == 0) return -1;
    const int at = __builtin_ctzll(past);
    int skip = u - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(own, at));
    uint32_t word = __builtin_amdgcn_readlane(w, at);
    for (; skip > 0; --skip) word &= word - 1;
    return 32 * at + __builtin_ctz(word);
}

// ids[first ..] == e for a token's `top` ids: the place of the first of them, or -1.
__device__ __forceinline__ int first_place(const int32_t *ids, int first, int top, int e)
{
    int place = -1;
#pragma unroll 4
    for (int j = top - 1; j >= 0; --j) place = ids[first + j] == e ? first + j : place;
    return place;
}

// The u-th expert that the tokens name and, in `list`, the places (token * top + first
// j) of the tokens that name it, in order.  -1: there are fewer experts.
struct Routing {
    uint32_t bits[MAX_EXPERTS / 32];
    int counts[MOE_MAX_TOKENS / 64];
    int list[MOE_MAX_TOKENS];
};

template <int WV, bool MANY>
__device__ __forceinline__ int route(const MoeArgs &p, int u, Routing &r, int &count, int tid, int lane, int wave)
{
    mark_experts<WV>(p.ids, p.tokens * p.top, p.experts, r.bits, tid);
    const int expert = expert_at(r.bits, u, lane);
    if (expert < 0) return -1;   // all waves alike
    // tokens in groups of 64, one per lane
    const int groups = MANY ? (p.tokens + 63) / 64 : 1;
    auto place_of = [&](int g) {
        const int t = 64 * g + lane;
        return t < p.tokens ? first_place(p.ids, t * p.top, p.top, expert) : -1;
    };
    int place[MANY ? MOE_MAX_TOKENS / 64 / WV : 1];
    if (MANY || wave == 0) {
#pragma unroll
        for (int i = 0; i < (MANY ? MOE_MAX_TOKENS / 64 / WV : 1); ++i) {
            const int g = wave + WV * i;
            place[i] = g < groups ? place_of(g) : -1;
            const uint64_t mine = __ballot(place[i] >= 0);
            if (lane == 0 && g < groups) r.counts[g] = __builtin_popcountll(mine);
        }
    }
    if (MANY) __syncthreads();
    if (MANY || wave == 0) {
#pragma unroll
        for (int i = 0; i < (MANY ? MOE_MAX_TOKENS / 64 / WV : 1); ++i) {
            int before = 0;
            for (int g = 0; MANY && g < min(groups, wave + WV * i); ++g) before += r.counts[g];
            const uint64_t mine = __ballot(place[i] >= 0);
            if (place[i] >= 0) r.list[before + lanes_below(mine)] = place[i];
        }
    }
    __syncthreads();
    count = 0;
    for (int g = 0; g < groups; ++g) count += r.counts[g];
    count = __builtin_amdgcn_readfirstlane(count);
    return expert;
}

// ------------------------------------------------------------ first product --

// h as the second product reads it; bf16 as the sum of two bf16 values (16 bits of it:
// one would add as much to y's error as its own rounding does; the second product
// waits for its weights, not for the matrix cores).
template <bool BF16>
__device__ __forceinline__ void store_h(const MoeArgs &p, int64_t at, float h)
{
    if constexpr (BF16) {
        uint16_t *out = static_cast<uint16_t *>(p.h);
        const uint16_t hi = f32_to_bf16_rne(h);
        const float rest = h - __uint_as_float((uint32_t)hi << 16);
        out[at] = hi;
        out[p.h_plane + at] = f32_to_bf16_rne(fabsf(rest) < __builtin_inff() ? rest : 0.0f);   // infinity has none
    } else {
        static_cast<float *>(p.h)[at] = h;
    }
}

// h of one expert's tokens, a strip of columns.
template <int WV, bool BF16, bool T, int W, int P, bool MANY>
__global__ void __launch_bounds__(64 * WV, 2) moe_up_kernel(MoeArgs p)
{
    __shared__ Routing routing;
    __shared__ float sums[WV / 2 * 16 * (MANY ? 4 : 1) * 16 * W * P];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int at = place_of_block<T>(p.max_used * p.strips_up);
    if (at < 0) return;
    const int u = at / p.strips_up, n0 = at % p.strips_up * 16 * W;
    int count;
    const int expert = route<WV, MANY>(p, u, routing, count, tid, lane, wave);
    if (expert < 0) return;
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    const In *w = static_cast<const In *>(p.up) + expert * p.stride_up;
    auto tile = [&](auto rt_c, auto u_c, int row0, int rows) {
        const int *list = routing.list + row0;
        product<WV, BF16, T, W, P, 1, decltype(rt_c)::value, decltype(u_c)::value>(
            w, p.ldup, p.inner, p.hidden, n0, p.x, 0, rows,
            [&](int r) { return (int64_t)(list[r] / p.top) * p.ldx; }, sums, lane, wave,
            [&](int r, int col, const float (&z)[P]) {
                float g[1] = {z[0]};
                act_apply<1>(p.act, false, g);
                const float h = P == 2 ? g[0] * z[P - 1] : g[0];
                store_h<BF16>(p, list[r] * p.ldh + n0 + col, h);
            });
    };
    using std::integral_constant;
    constexpr int STEPS = 8 / (W * P);   // per pass
    if constexpr (!MANY) {
        tile(integral_constant<int, 1>(), integral_constant<int, STEPS>(), 0, count);
    } else {
        for (int row0 = 0; row0 < count; row0 += 64) {
            const int rows = min(64, count - row0);
            if (row0 > 0) __syncthreads();   // the sums of the rows before are read
            if (rows <= 16)
                tile(integral_constant<int, 1>(), integral_constant<int, T ? STEPS : 1>(), row0, rows);
            else if (rows <= 32)
                tile(integral_constant<int, 2>(), integral_constant<int, T ? 2 : 1>(), row0, rows);
            else
                tile(integral_constant<int, 4>(), integral_constant<int, 1>(), row0, rows);
        }
    }
}

// ------------------------------------------- second product, up to 16 tokens --

// y of all tokens, a strip of columns: the block goes through all experts (or through
// its part of them), each expert's inner width in passes; the list of (expert, whole
// pass) is cut into one run per wave, then the waves take the experts' cut passes in
// turn.  A wave adds an expert's sums, weighted, to its own y in LDS when it leaves
// the expert; the waves' y are added at the end, in order.
struct Entry {
    int place;       // token * top + the first j that names the expert
    float weight;    // all its weights
};

template <bool BF16, bool T, int W, int U>
__device__ __forceinline__ void down_strip(const MoeArgs &p, int n0, const uint16_t *experts, const int32_t *ids,
                                           const float *weights, Entry (*lists)[16], float *y, int begin, int end,
                                           int cut, int cuts, int step, int lane)
{
    using S = Strip<BF16, T, W, 1, BF16 ? 2 : 1, 1, U>;
    using In = typename S::In;
    const int passes = p.inner / S::KP;   // whole ones
    S s;
    s.place(lane, n0, p.hidden, p.inner, p.lddown);
    s.x_plane = p.h_plane;
    floatx4 acc[W][1];
    clear(acc);
    // the rows and weights of the u-th expert, its list in buffer b; lane t looks after token t
    auto enter = [&](int u, int b) {
        const int e = __builtin_amdgcn_readfirstlane(experts[u]);
        s.w = static_cast<const In *>(p.down) + e * p.stride_down;
        int place = -1;
        float weight = 0.0f;
        if (lane < p.tokens) {
#pragma unroll 4
            for (int j = p.top - 1; j >= 0; --j) {
                const bool here = ids[lane * p.top + j] == e;
                place = here ? lane * p.top + j : place;
                weight += here ? weights[lane * p.top + j] : 0.0f;
            }
        }
        const uint64_t mine = __ballot(place >= 0);
        if (place >= 0) lists[b][lanes_below(mine)] = Entry{place, weight};
        wave_order();
        const int n = __builtin_popcountll(mine);
        s.xr[0] = static_cast<const In *>(p.h) + (int64_t)lists[b][min(s.c, n - 1)].place * p.ldh;
        return n;
    };
    auto leave = [&](int b, int count) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 4 * s.q + r;
            if (row >= count) continue;
            const Entry at = lists[b][row];
            float *out = y + at.place / p.top * (16 * W);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int col = s.column(j);
                // (pieces that N's end moved back repeat columns of others)
                if (T || col >= W * s.c) out[col] += at.weight * acc[j][0][r];
            }
        }
        clear(acc);
        wave_order();
    };
    typename S::Regs cur, nxt;
    if (begin < end) {
        int u = begin / passes, pass = begin - u * passes, b = 0;
        const int rot = n0 / (16 * W) % passes;   // as in product()
        auto k_of = [&](int pass) {
            const int at = pass + rot;
            return (at >= passes ? at - passes : at) * S::KP;
        };
        int count = enter(u, b), next_count = 0;
        s.template load<false>(k_of(pass), cur);
        for (int i = begin; i < end; ++i) {
            bool last = true;
            if (i + 1 < end) {
                last = ++pass == passes;
                if (last) {
                    pass = 0;
                    next_count = enter(++u, b ^ 1);
                }
                s.template load<false>(k_of(pass), nxt);
            }
            s.compute(cur, acc);
            if (last) {
                leave(b, count);
                b ^= 1;
                count = next_count;
            }
            cur = nxt;
        }
    }
    if (passes * S::KP < p.inner)
        for (int u = cut; u < cuts; u += step) {
            const int count = enter(u, 0);
            s.template load<true>(passes * S::KP, cur);
            s.compute(cur, acc);
            leave(0, count);
        }
}

template <bool BF16, bool T, int W>
__global__ void __launch_bounds__(512) moe_down_few_kernel(MoeArgs p)
{
    constexpr int WV = 8, BN = 16 * W, U = 4 / W, KP = U * 4 * (BF16 ? 8 : 4);
    __shared__ uint32_t bits[MAX_EXPERTS / 32];
    __shared__ uint16_t experts[16 * MOE_MAX_TOP];
    __shared__ int32_t ids[16 * MOE_MAX_TOP];
    __shared__ float weights[16 * MOE_MAX_TOP];
    __shared__ Entry lists[WV][2][16];
    __shared__ float y[WV][16 * BN];
    __shared__ int shared_used;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int at = place_of_block<T>(p.strips_down * p.parts);
    if (at < 0) return;
    const int n0 = at % p.strips_down * BN, part = at / p.strips_down, places = p.tokens * p.top;

    for (int i = tid; i < places; i += 64 * WV) {
        ids[i] = p.ids[i];
        weights[i] = p.weights[i];
    }
    for (int i = tid; i < WV * 16 * BN; i += 64 * WV) (&y[0][0])[i] = 0.0f;
    mark_experts<WV>(p.ids, places, p.experts, bits, tid);
    if (wave == 0) {
        uint32_t w = lane < MAX_EXPERTS / 32 ? bits[lane] : 0;
        const int own = __builtin_popcount(w), upto = scan(own, lane);
        for (int i = upto - own; w != 0; ++i, w &= w - 1) experts[i] = (uint16_t)(32 * lane + __builtin_ctz(w));
        if (lane == 63) shared_used = upto;
    }
    __syncthreads();
    const int used = shared_used, passes = p.inner / KP;
    const int64_t items = (int64_t)used * passes;
    const int64_t first = items * part / p.parts, last = items * (part + 1) / p.parts;
    const int begin = (int)(first + (last - first) * wave / WV), end = (int)(first + (last - first) * (wave + 1) / WV);
    down_strip<BF16, T, W, U>(p, n0, experts, ids, weights, lists[wave], y[wave], begin, end, part * WV + wave, used,
                               p.parts * WV, lane);
    __syncthreads();
    for (int i = tid; i < p.tokens * BN; i += 64 * WV) {
        const int token = i / BN, col = n0 + i % BN;
        if (col >= p.hidden) continue;
        float v[1] = {0.0f};
#pragma unroll
        for (int w = 0; w < WV; ++w) v[0] += y[w][i];
        if (p.parts > 1) {
            p.ws[((int64_t)part * p.tokens + token) * p.hidden + col] = v[0];
        } else {
            const float none[1] = {0.0f};
            finish_piece<1>(p.e, 0, token, col, 1, none, v);
        }
    }
}

// y of parts: their sums in order.
__global__ void __launch_bounds__(256) moe_join_kernel(MoeArgs p)
{
    const int64_t total = (int64_t)p.tokens * p.hidden;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t token = i / p.hidden;
        float v[1] = {0.0f};
        const float none[1] = {0.0f};
        for (int k = 0; k < p.parts; ++k) v[0] += p.ws[k * total + i];
        finish_piece<1>(p.e, 0, token, (int)(i - token * p.hidden), 1, none, v);
    }
}

// --------------------------------------------- second product, more tokens --

// One expert's rows, a strip of columns, to ws by place.
template <int WV, bool BF16, bool T, int W>
__global__ void __launch_bounds__(64 * WV, 2) moe_down_rows_kernel(MoeArgs p)
{
    __shared__ Routing routing;
    __shared__ float sums[WV / 2 * 64 * 16 * W];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int at = place_of_block<T>(p.max_used * p.strips_down);
    if (at < 0) return;
    const int u = at / p.strips_down, n0 = at % p.strips_down * 16 * W;
    int count;
    const int expert = route<WV, true>(p, u, routing, count, tid, lane, wave);
    if (expert < 0) return;
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    const In *w = static_cast<const In *>(p.down) + expert * p.stride_down;
    auto tile = [&](auto rt_c, auto u_c, int row0, int rows) {
        const int *list = routing.list + row0;
        product<WV, BF16, T, W, 1, BF16 ? 2 : 1, decltype(rt_c)::value, decltype(u_c)::value>(
            w, p.lddown, p.hidden, p.inner, n0, p.h, p.h_plane, rows, [&](int r) { return (int64_t)list[r] * p.ldh; },
            sums, lane, wave,
            [&](int r, int col, const float (&z)[1]) { p.ws[(int64_t)list[r] * p.hidden + n0 + col] = z[0]; });
    };
    using std::integral_constant;
    for (int row0 = 0; row0 < count; row0 += 64) {
        const int rows = min(64, count - row0);
        if (row0 > 0) __syncthreads();   // the sums of the rows before are read
        if (rows <= 16)
            tile(integral_constant<int, 1>(), integral_constant<int, T ? 8 / W : 1>(), row0, rows);
        else if (rows <= 32)
            tile(integral_constant<int, 2>(), integral_constant<int, T ? 2 : 1>(), row0, rows);
        else
            tile(integral_constant<int, 4>(), integral_constant<int, 1>(), row0, rows);
    }
}

// y of a token from its experts' rows, in the order of its ids; a block has 256
// columns of a token.
__global__ void __launch_bounds__(256) moe_sum_kernel(MoeArgs p, int col_blocks)
{
    __shared__ int32_t ids[MOE_MAX_TOP];
    __shared__ float weights[MOE_MAX_TOP], shares[MOE_MAX_TOP];
    __shared__ int counts[MOE_MAX_TOP];   // whether a place counts: an expert's first
    const int tid = (int)threadIdx.x, token = (int)blockIdx.x / col_blocks;
    const int col = ((int)blockIdx.x - token * col_blocks) * 256 + tid;
    if (tid < p.top) {
        ids[tid] = p.ids[token * p.top + tid];
        weights[tid] = p.weights[token * p.top + tid];
    }
    __syncthreads();
    if (tid < p.top) {
        // all the weights of an expert at its first place
        bool first = (unsigned)ids[tid] < (unsigned)p.experts;
        float sum = 0.0f;
        for (int j = p.top - 1; j >= 0; --j)
            if (ids[j] == ids[tid]) {
                sum += weights[j];
                if (j < tid) first = false;
            }
        shares[tid] = sum;
        counts[tid] = first;
    }
    __syncthreads();
    if (col >= p.hidden) return;
    float v[1] = {0.0f};
    const float none[1] = {0.0f};
    for (int j = 0; j < p.top; ++j)
        if (counts[j]) v[0] += shares[j] * p.ws[((int64_t)token * p.top + j) * p.hidden + col];
    finish_piece<1>(p.e, 0, token, col, 1, none, v);
}

// ------------------------------------------------------------ small widths --

// Widths below 8, which the vectors above do not fit: a thread per value.
template <bool BF16>
__device__ __forceinline__ float value(const void *x, int64_t at)
{
    return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(x)[at] << 16) : static_cast<const float *>(x)[at];
}

template <bool BF16, bool T>
__global__ void __launch_bounds__(256) moe_small_up_kernel(MoeArgs p)
{
    const int64_t total = (int64_t)p.tokens * p.top * p.inner;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int place = (int)(i / p.inner), col = (int)(i - (int64_t)place * p.inner), token = place / p.top;
        const int e = p.ids[place];
        if ((unsigned)e >= (unsigned)p.experts) continue;
        float z[2] = {0.0f, 0.0f};
        for (int k = 0; k < p.hidden; ++k) {
            const float x = value<BF16>(p.x, token * p.ldx + k);
            for (int f = 0; f < (p.gated ? 2 : 1); ++f) {
                const int n = f * p.inner + col;
                z[f] += x * value<BF16>(p.up, e * p.stride_up + (T ? n * p.ldup + k : k * p.ldup + n));
            }
        }
        float g[1] = {z[0]};
        act_apply<1>(p.act, false, g);
        store_h<BF16>(p, place * p.ldh + col, p.gated ? g[0] * z[1] : g[0]);
    }
}

template <bool BF16, bool T>
__global__ void __launch_bounds__(256) moe_small_down_kernel(MoeArgs p)
{
    const int64_t total = (int64_t)p.tokens * p.top * p.hidden;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int place = (int)(i / p.hidden), col = (int)(i - (int64_t)place * p.hidden);
        const int e = p.ids[place];
        if ((unsigned)e >= (unsigned)p.experts) continue;
        float sum = 0.0f;
        for (int k = 0; k < p.inner; ++k) {
            float h = value<BF16>(p.h, place * p.ldh + k);
            if (BF16) h += value<BF16>(p.h, p.h_plane + place * p.ldh + k);
            sum += h * value<BF16>(p.down, e * p.stride_down + (T ? col * p.lddown + k : k * p.lddown + col));
        }
        p.ws[i] = sum;
    }
}

// ------------------------------------------------------------------ launch --

// Fragments of 16 columns of a block, both panels of the first product.
constexpr int strip(bool t, bool wide) { return t ? (wide ? 4 : 2) : (wide ? 8 : 4); }
// Waves of a block.  With more than 16 tokens the waves' registers leave room for 8 of
// them on a unit either way; blocks of 4 overlap one another's start and end (64
// tokens, 64 experts of 2048 x 1024: 186 us, with blocks of 8 200).
constexpr int WAVES_FEW = 8, WAVES_MANY = 4;

template <bool BF16, bool T, int P>
void (*up_kernel(const MoePlan &plan))(MoeArgs)
{
    constexpr int WIDE = strip(T, true) / P, NARROW = strip(T, false) / P;
    constexpr int NARROW_MANY = T ? WIDE : NARROW;   // N x K weights: always wide
    return plan.many ? (plan.wide_up ? moe_up_kernel<WAVES_MANY, BF16, T, WIDE, P, true>
                                     : moe_up_kernel<WAVES_MANY, BF16, T, NARROW_MANY, P, true>)
                     : (plan.wide_up ? moe_up_kernel<WAVES_FEW, BF16, T, WIDE, P, false>
                                     : moe_up_kernel<WAVES_FEW, BF16, T, NARROW, P, false>);
}

hipError_t run(void (*kernel)(MoeArgs), int64_t blocks, int threads, const MoeArgs &a, hipStream_t stream)
{
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), 0, stream, a);
    return hipGetLastError();
}

template <bool BF16, bool T>
hipError_t launch(const MoeArgs &a, const MoePlan &plan, hipStream_t stream)
{
    const int threads = 64 * (plan.many ? WAVES_MANY : WAVES_FEW);
    auto up = plan.small  ? moe_small_up_kernel<BF16, T>
              : a.gated   ? up_kernel<BF16, T, 2>(plan)
                          : up_kernel<BF16, T, 1>(plan);
    hipError_t err = run(up, plan.blocks_up, plan.small ? 256 : threads, a, stream);
    if (err != hipSuccess) return err;
    constexpr int WIDE = strip(T, true), NARROW = strip(T, false), NARROW_MANY = T ? WIDE : NARROW;
    auto down = plan.small       ? moe_small_down_kernel<BF16, T>
                : plan.many      ? (plan.wide_down ? moe_down_rows_kernel<WAVES_MANY, BF16, T, WIDE>
                                                   : moe_down_rows_kernel<WAVES_MANY, BF16, T, NARROW_MANY>)
                : plan.wide_down ? moe_down_few_kernel<BF16, T, WIDE / 2>
                                 : moe_down_few_kernel<BF16, T, NARROW / 2>;
    err = run(down, plan.blocks_down, plan.small ? 256 : threads, a, stream);
    if (err != hipSuccess) return err;
    if (plan.many || plan.small) {
        const int col_blocks = (a.hidden + 255) / 256;
        hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)(a.tokens * col_blocks)), dim3(256), 0, stream, a, col_blocks);
        return hipGetLastError();
    }
    if (a.parts == 1) return hipSuccess;
    const int64_t blocks = ((int64_t)a.tokens * a.hidden + 255) / 256;
    return run(moe_join_kernel, blocks < 65536 ? blocks : 65536, 256, a, stream);
}

}  // namespace

// Columns of a block of the first product, and of the second.
int moe_strip_up(bool t, bool gated, bool wide) { return 16 * strip(t, wide) / (gated ? 2 : 1); }
int moe_strip_down(bool t, bool many, bool wide) { return (many ? 16 : 8) * strip(t, wide); }

hipError_t launch_moe(const MoeArgs &a, const MoePlan &plan, bool bf16, bool transw, hipStream_t stream)
{
    return bf16 ? (transw ? launch<true, true>(a, plan, stream) : launch<true, false>(a, plan, stream))
                : (transw ? launch<false, true>(a, plan, stream) : launch<false, false>(a, plan, stream));
}

}  // namespace dg
