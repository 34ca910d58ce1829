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
// Tokens are taken in chunks of 16, 32 or 64, rows of 16 x 16 MFMAs.  A token that
// names an expert twice is one row with both its weights.
#include "linear_kernel.hpp"
#include "serving.hpp"

namespace dg {
namespace {

constexpr int WV = 8;   // waves of a block

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
    using F = FewRows<BF16, T ? 1 : 0, W, WV>;   // its loads and products
    using In = typename F::In;
    static constexpr int KV = F::KV, STEP = 4 * KV, KP = U * STEP;
    struct Regs {
        u32x4 x[U][XP][RT];
        u32x4 w[T ? U * P * W : 1];
        uint32_t v[T ? 1 : U * P * KV][T ? 1 : F::PD];
    };

    const In *xr[RT];    // this lane's rows of x
    int64_t x_plane;     // elements from a plane to the next
    const In *w;
    int64_t ldw;
    int q, c, n0, N, K;

    __device__ __forceinline__ int first_col() const { return min(n0 + W * c, max(N - W, 0)); }

    template <bool TAIL, bool NARROW>
    __device__ __forceinline__ void load(int k0, Regs &r) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u * STEP + q * KV;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if constexpr (T) {
#pragma unroll
                    for (int f = 0; f < W; ++f) {
                        const In *row = w + (int64_t)(p * N + min(n0 + 16 * f + c, N - 1)) * ldw;
                        r.w[(u * P + p) * W + f] = TAIL ? F::load_masked(row, k, K) : F::load_chunk(row + k);
                    }
                } else {
                    const int col = first_col();
#pragma unroll
                    for (int i = 0; i < KV; ++i) {
                        const In *row = w + (int64_t)(TAIL ? min(k + i, K - 1) : k + i) * ldw + p * (int64_t)N;
                        union {
                            typename F::piece v;
                            In e[W];
                            uint32_t d[F::PD];
                        } t;
                        if constexpr (NARROW) {
#pragma unroll
                            for (int j = 0; j < W; ++j) t.e[j] = row[min(col + j, N - 1)];
                        } else {
                            t.v = *reinterpret_cast<const typename F::piece *>(row + col);
                        }
#pragma unroll
                        for (int d = 0; d < F::PD; ++d)
                            r.v[(u * P + p) * KV + i][d] = !TAIL || k + i < K ? t.d[d] : 0u;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int h = 0; h < XP; ++h)
                    r.x[u][h][t] = TAIL ? F::load_masked(xr[t] + h * x_plane, k, K) : F::load_chunk(xr[t] + h * x_plane + k);
        }
    }
    // The pass at k0 < K, whole or cut.
    template <bool NARROW>
    __device__ __forceinline__ void load(int k0, Regs &r) const
    {
        if (k0 + KP <= K)
            load<false, NARROW>(k0, r);
        else
            load<true, NARROW>(k0, r);
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

// ------------------------------------------------------- experts and tokens --

// The set of experts that a chunk's ids name: a bit each, by one wave.
constexpr int MAX_EXPERTS = MOE_MAX_EXPERTS;

__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void mark_experts(const int32_t *ids, int count, int experts, uint32_t *bits, int lane)
{
    if (lane < MAX_EXPERTS / 32) bits[lane] = 0;
    wave_order();
    for (int i = lane; i < count; i += 64) {
        const unsigned e = (unsigned)ids[i];
        if (e < (unsigned)experts) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    wave_order();
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

struct Place {
    int slot;        // t * top + the first j that names the expert
    float weight;    // all its weights
};

// The tokens of a chunk that name expert e, in order: their places, and how many.
// Lane t looks after token t.
template <bool WEIGHTS, class Ids, class Weights>
__device__ __forceinline__ int list_tokens(int e, int tokens, int top, Ids &&id, Weights &&weight, Place *list, int lane)
{
    int slot = -1;
    float sum = 0.0f;
    if (lane < tokens)
        for (int j = top - 1; j >= 0; --j)
            if (id(lane * top + j) == e) {
                slot = lane * top + j;
                if (WEIGHTS) sum += weight(slot);
            }
    const uint64_t mine = __ballot(slot >= 0);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(mine >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mine, 0));
    if (slot >= 0) list[before] = Place{slot, sum};
    wave_order();
    return __builtin_popcountll(mine);
}

// ------------------------------------------------------------ first product --

// h of one expert's tokens of a chunk, a strip of columns over the whole of the
// hidden width; the waves take turns along it, and their sums meet in LDS.  h is
// stored as the second product reads it; bf16 as the sum of two bf16 values (16 bits
// of it: one would add as much to y's error as its own rounding does; the second
// product waits for its weights, not for the matrix cores).
template <bool BF16, bool T, int W, int P, int RT, int U>
__device__ __forceinline__ void up_tile(const MoeArgs &p, int expert, int n0, int t0, int count, const Place *list,
                                        float *sums, int lane, int wave)
{
    using S = Strip<BF16, T, W, P, 1, RT, U>;
    using In = typename S::In;
    constexpr int BN = 16 * W * P, ROWS = 16 * RT;
    S s;
    s.q = lane >> 4;
    s.c = lane & 15;
    s.n0 = n0;
    s.N = p.inner;
    s.K = p.hidden;
    s.ldw = p.ldup;
    s.w = static_cast<const In *>(p.up) + expert * p.stride_up;
    s.x_plane = 0;
#pragma unroll
    for (int t = 0; t < RT; ++t)
        s.xr[t] = static_cast<const In *>(p.x) + (int64_t)(t0 + list[min(16 * t + s.c, count - 1)].slot / p.top) * p.ldx;
    floatx4 acc[P * W][RT];
    clear(acc);
    auto run = [&](auto narrow_c) {
        constexpr bool NARROW = decltype(narrow_c)::value;
        typename S::Regs cur, nxt;
        int k = wave * S::KP;
        if (k < p.hidden) s.template load<NARROW>(k, cur);
        for (; k < p.hidden; k += WV * S::KP) {
            if (k + WV * S::KP < p.hidden) s.template load<NARROW>(k + WV * S::KP, nxt);
            s.compute(cur, acc);
            cur = nxt;
        }
    };
    if (T || p.inner >= W)
        run(std::false_type());
    else
        run(std::true_type());
#pragma unroll
    for (int f = 0; f < P * W; ++f) {
        const int col = s.column(f % W);
        if (T || col >= 0)
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sums[(wave * ROWS + 16 * t + 4 * s.q + r) * BN + f / W * 16 * W + col] = acc[f][t][r];
    }
    __syncthreads();
    for (int id = (int)threadIdx.x; id < count * 16 * W; id += 64 * WV) {
        const int row = id / (16 * W), col = id % (16 * W);
        if (n0 + col >= p.inner) continue;
        float z[P];
#pragma unroll
        for (int f = 0; f < P; ++f) {
            z[f] = 0.0f;
#pragma unroll
            for (int v = 0; v < WV; ++v) z[f] += sums[(v * ROWS + row) * BN + f * 16 * W + col];
        }
        float g[1] = {z[0]};
        act_apply<1>(p.act, false, g);
        const float h = P == 2 ? g[0] * z[P - 1] : g[0];
        const int64_t at = ((int64_t)t0 * p.top + list[row].slot) * p.ldh + n0 + col;
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
}

template <bool BF16, bool T, int P, int RTMAX>
struct UpShape {
    static constexpr int W = (T ? 2 : 4) / P;
    static constexpr int LDS = WV * 16 * RTMAX * 16 * W * P;   // floats
};

template <bool BF16, bool T, int P, int RTMAX>
__global__ void __launch_bounds__(64 * WV) moe_up_kernel(MoeArgs p)
{
    using Shape = UpShape<BF16, T, P, RTMAX>;
    constexpr int W = Shape::W;
    __shared__ uint32_t bits[WV][MAX_EXPERTS / 32];
    __shared__ Place list[WV][64];
    __shared__ float sums[Shape::LDS];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int strip = (int)blockIdx.x % p.strips_up, rest = (int)blockIdx.x / p.strips_up;
    const int u = rest % p.max_used, chunk = rest / p.max_used;
    const int t0 = chunk * 16 * RTMAX, tokens = min(16 * RTMAX, p.tokens - t0);
    const int32_t *ids = p.ids + (int64_t)t0 * p.top;

    // each wave for itself, without a barrier
    mark_experts(ids, tokens * p.top, p.experts, bits[wave], lane);
    const int expert = expert_at(bits[wave], u, lane);
    if (expert < 0) return;   // all waves alike
    const int count = list_tokens<false>(expert, tokens, p.top, [&](int i) { return ids[i]; },
                                         [](int) { return 0.0f; }, list[wave], lane);
    const int n0 = strip * 16 * W;
    if (RTMAX == 1 || count <= 16)
        up_tile<BF16, T, W, P, 1, 4>(p, expert, n0, t0, count, list[wave], sums, lane, wave);
    else if (RTMAX == 2 || count <= 32)
        up_tile<BF16, T, W, P, RTMAX < 2 ? 1 : 2, 2>(p, expert, n0, t0, count, list[wave], sums, lane, wave);
    else
        up_tile<BF16, T, W, P, RTMAX < 4 ? 1 : 4, 2>(p, expert, n0, t0, count, list[wave], sums, lane, wave);
}

// ----------------------------------------------------------- second product --

// y of a chunk's tokens, a strip of columns: the block goes through all experts of
// the chunk (or through its part of them), each expert's inner width in passes; the
// list of (expert, pass) is cut into one run per wave.  A wave adds an expert's
// sums, weighted, to its own y in LDS when it leaves the expert; the waves' y are
// added at the end, in order.
template <bool BF16, bool T, int W, int RT, int U, int NT>
__device__ __forceinline__ void down_strip(const MoeArgs &p, int n0, int t0, int tokens, const uint16_t *experts,
                                           const int32_t *ids, const float *weights, Place (*lists)[64], float *y,
                                           int begin, int end, int passes, int lane)
{
    using S = Strip<BF16, T, W, 1, BF16 ? 2 : 1, RT, U>;
    using In = typename S::In;
    S s;
    s.q = lane >> 4;
    s.c = lane & 15;
    s.n0 = n0;
    s.N = p.hidden;
    s.K = p.inner;
    s.ldw = p.lddown;
    s.x_plane = p.h_plane;
    if (begin >= end) return;
    floatx4 acc[W][RT];
    clear(acc);
    int u = begin / passes, pass = begin - u * passes;
    int which = 0, count = 0, next_count = 0;
    // the rows and weights of the u-th expert, its list in buffer b
    auto enter = [&](int b) {
        const int e = experts[u];
        s.w = static_cast<const In *>(p.down) + e * p.stride_down;
        const int n = list_tokens<true>(e, tokens, p.top, [&](int i) { return ids[i]; },
                                        [&](int i) { return weights[i]; }, lists[b], lane);
#pragma unroll
        for (int t = 0; t < RT; ++t)
            s.xr[t] = static_cast<const In *>(p.h) +
                      ((int64_t)t0 * p.top + lists[b][min(16 * t + s.c, n - 1)].slot) * p.ldh;
        return n;
    };
    auto run = [&](auto narrow_c) {
        constexpr bool NARROW = decltype(narrow_c)::value;
        typename S::Regs cur, nxt;
        count = enter(which);
        s.template load<NARROW>(pass * S::KP, cur);
        for (int i = begin; i < end; ++i) {
            bool leave = true;
            if (i + 1 < end) {
                leave = ++pass == passes;
                if (leave) {
                    pass = 0;
                    ++u;
                    next_count = enter(which ^ 1);
                }
                s.template load<NARROW>(pass * S::KP, nxt);
            }
            s.compute(cur, acc);
            if (leave) {
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 16 * t + 4 * s.q + r;
                        if (row >= count) continue;
                        const Place at = lists[which][row];
                        float *out = y + at.slot / p.top * (16 * W);
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            const int col = s.column(j);
                            // (pieces that N's end moved back repeat columns of others)
                            if (T || col >= W * s.c) out[col] += at.weight * acc[j][t][r];
                        }
                    }
                clear(acc);
                which ^= 1;
                count = next_count;
                wave_order();
            }
            cur = nxt;
        }
    };
    if (T || p.hidden >= W)
        run(std::false_type());
    else
        run(std::true_type());
}

template <bool BF16, bool T, int RTMAX>
struct DownShape {
    static constexpr int W = RTMAX == 1 && T ? 1 : 2;
};

template <bool BF16, bool T, int RTMAX>
__global__ void __launch_bounds__(64 * WV) moe_down_kernel(MoeArgs p)
{
    constexpr int W = DownShape<BF16, T, RTMAX>::W, NT = 16 * RTMAX, BN = 16 * W;
    __shared__ uint32_t bits[MAX_EXPERTS / 32];
    __shared__ uint16_t experts[MAX_EXPERTS];
    __shared__ int32_t ids[NT * MOE_MAX_TOP];
    __shared__ float weights[NT * MOE_MAX_TOP];
    __shared__ Place lists[WV][2][64];
    __shared__ float y[WV][NT * BN];
    __shared__ int counts[RTMAX > 1 ? MAX_EXPERTS : 1];
    __shared__ int shared_used, shared_most;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int strip = (int)blockIdx.x % p.strips_down, rest = (int)blockIdx.x / p.strips_down;
    const int part = rest % p.parts, chunk = rest / p.parts;
    const int t0 = chunk * NT, tokens = min(NT, p.tokens - t0), slots = tokens * p.top;

    for (int i = tid; i < slots; i += 64 * WV) {
        ids[i] = p.ids[(int64_t)t0 * p.top + i];
        weights[i] = p.weights[(int64_t)t0 * p.top + i];
    }
    for (int i = tid; i < WV * NT * BN; i += 64 * WV) (&y[0][0])[i] = 0.0f;
    if (RTMAX > 1)
        for (int i = tid; i < MAX_EXPERTS; i += 64 * WV) counts[i] = 0;
    if (tid == 0) shared_most = 0;
    __syncthreads();
    if (wave == 0) {
        mark_experts(ids, slots, p.experts, bits, lane);
        uint32_t w = lane < MAX_EXPERTS / 32 ? bits[lane] : 0;
        const int own = __builtin_popcount(w), upto = scan(own, lane);
        for (int at = upto - own; w != 0; ++at, w &= w - 1) experts[at] = (uint16_t)(32 * lane + __builtin_ctz(w));
        if (lane == 63) shared_used = upto;
    } else if (RTMAX > 1) {
        for (int i = tid - 64; i < slots; i += 64 * (WV - 1))
            if ((unsigned)ids[i] < (unsigned)p.experts) {
                const int n = atomicAdd(&counts[ids[i]], 1) + 1;
                if (n > 16) atomicMax(&shared_most, n);
            }
    }
    __syncthreads();
    const int used = shared_used, most = shared_most;   // (most: 0 up to 16 rows; a token that names one twice counts twice)
    const int n0 = strip * BN;
    auto share = [&](auto u_c, auto rt_c) {
        constexpr int U = decltype(u_c)::value, RT = decltype(rt_c)::value;
        constexpr int KP = U * 4 * (BF16 ? 8 : 4);
        const int passes = (p.inner + KP - 1) / KP;
        const int64_t items = (int64_t)used * passes;
        const int64_t first = items * part / p.parts, last = items * (part + 1) / p.parts;
        const int begin = (int)(first + (last - first) * wave / WV), end = (int)(first + (last - first) * (wave + 1) / WV);
        down_strip<BF16, T, W, RT, U, NT>(p, n0, t0, tokens, experts, ids, weights, lists[wave], y[wave], begin, end,
                                          passes, lane);
    };
    if (RTMAX == 1 || most <= 16)
        share(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    else if (RTMAX == 2 || most <= 32)
        share(std::integral_constant<int, 2>(), std::integral_constant<int, RTMAX < 2 ? 1 : 2>());
    else
        share(std::integral_constant<int, 1>(), std::integral_constant<int, RTMAX < 4 ? 1 : 4>());
    __syncthreads();
    for (int i = tid; i < tokens * BN; i += 64 * WV) {
        const int token = i / BN, col = n0 + i % BN;
        if (col >= p.hidden) continue;
        float v[1] = {0.0f};
#pragma unroll
        for (int w = 0; w < WV; ++w) v[0] += y[w][i];
        if (p.parts > 1) {
            p.ws[((int64_t)part * p.tokens + t0 + token) * p.hidden + col] = v[0];
        } else {
            const float none[1] = {0.0f};
            finish_piece<1>(p.e, 0, t0 + token, col, 1, none, v);
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

template <bool BF16, bool T, int RTMAX>
hipError_t launch(const MoeArgs &a, const MoePlan &plan, hipStream_t stream)
{
    if (plan.blocks_up > 0) {
        auto kernel = a.gated ? moe_up_kernel<BF16, T, 2, RTMAX> : moe_up_kernel<BF16, T, 1, RTMAX>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)plan.blocks_up), dim3(64 * WV), 0, stream, a);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL((moe_down_kernel<BF16, T, RTMAX>), dim3((unsigned)plan.blocks_down), dim3(64 * WV), 0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.parts == 1) return err;
    const int64_t blocks = ((int64_t)a.tokens * a.hidden + 255) / 256;
    hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <bool BF16, bool T>
hipError_t launch(const MoeArgs &a, const MoePlan &plan, hipStream_t stream)
{
    return plan.rows == 16   ? launch<BF16, T, 1>(a, plan, stream)
           : plan.rows == 32 ? launch<BF16, T, 2>(a, plan, stream)
                             : launch<BF16, T, 4>(a, plan, stream);
}

}  // namespace

int moe_strip_up(bool t, bool gated)
{
    return 16 * (gated ? (t ? UpShape<true, true, 2, 1>::W : UpShape<true, false, 2, 1>::W)
                       : (t ? UpShape<true, true, 1, 1>::W : UpShape<true, false, 1, 1>::W));
}
int moe_strip_down(bool t, int rows)
{
    return 16 * (rows == 16 ? (t ? DownShape<true, true, 1>::W : DownShape<true, false, 1>::W)
                            : (t ? DownShape<true, true, 2>::W : DownShape<true, false, 2>::W));
}

hipError_t launch_moe(const MoeArgs &a, const MoePlan &plan, bool bf16, bool transw, hipStream_t stream)
{
    return bf16 ? (transw ? launch<true, true>(a, plan, stream) : launch<true, false>(a, plan, stream))
                : (transw ? launch<false, true>(a, plan, stream) : launch<false, false>(a, plan, stream));
}

}  // namespace dg
