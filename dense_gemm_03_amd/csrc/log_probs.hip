// Log probabilities of given tokens, entropy and alternatives, and their gradient.
//
//     m = max z     c = fl(a m),  a = scale log2(e)     t_j = a z_j - c     s = sum 2^t_j     u = sum t_j 2^t_j
//     L = ln s - ln2 (a m - c)     entropy = ln s - ln2 u / s     logprob = scale (z_token - m) - L
//
// t_j is one fused multiply-add; what c lacks of a m is the same for all terms and
// known exactly (a m - c is another), so a large m costs no digits.
//
// One pass over the logits: each lane keeps (m, s, u) of what it has read and moves
// them to a larger m when it finds one, 32 logits at a time, which are loaded while the
// 32 before are summed.
//
// Bound by HBM and by the exponents' arithmetic alike with many rows (4001 x 50021 bf16, 5
// alternatives: 84 us, 4.7 TB/s), by latency with few: 1 x 131072 fp32 takes 4.7 us for the
// parts and 2.8 us to join them, with 20 alternatives 9.7 and 5.5.
#include "serving.hpp"
#include "topk.hpp"

namespace dg {
namespace {

constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
constexpr float kLowest = -3.402823466e38f;
constexpr int CHUNK = 64 * 32;   // logits per wave and step: 32 per lane

// Below 2^-200 nothing is left in fp32: exponents are bounded there where they are
// multiplied, so that a forbidden place (t = -infinity) adds 0 and not NaN.
__device__ __forceinline__ float bounded(float t) { return fmaxf(t, -200.0f); }

// Whether a m is so large that what c lacks of it, half a unit, may be an exponent of
// more than 1/2.  Distances are then formed before they are scaled, and c is a m itself.
__device__ __forceinline__ bool huge(float m, float a) { return !(fabsf(a * m) < 16777216.0f); }
// a m - c
__device__ __forceinline__ float lacking(float m, float a)
{
    const float c = a * m;
    return huge(m, a) ? 0.0f : __builtin_fmaf(a, m, -c);
}

struct Sums {
    float m = kLowest, s = 0.0f, u = 0.0f;   // m is a number even where nothing or -infinity was read

    // to the larger maximum `to`
    __device__ __forceinline__ void move(float to, float a)
    {
#pragma clang fp contract(off)   // a m and a to are the c's that the sums were formed with
        const float t = bounded(huge(m, a) || huge(to, a) ? a * (m - to) - lacking(m, a) + lacking(to, a) : a * m - a * to);
        const float f = __builtin_amdgcn_exp2f(t);
        u = __builtin_fmaf(s, t, u) * f;
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void add(Sums o, float a)
    {
        const float to = fmaxf(m, o.m);
        move(to, a);
        o.move(to, a);
        s += o.s;
        u += o.u;
    }
    __device__ __forceinline__ void add_lanes(float a)   // of all 64
    {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            add(Sums{__shfl_xor(m, d), __shfl_xor(s, d), __shfl_xor(u, d)}, a);
        }
    }
};

template <bool BF16>
__device__ __forceinline__ float logit_at(const void *logits, int64_t at)
{
    return BF16 ? __uint_as_float((uint32_t) static_cast<const uint16_t *>(logits)[at] << 16)
                : static_cast<const float *>(logits)[at];
}

// What a row's sums come to, written by one wave.
template <bool BF16>
__device__ __forceinline__ void finish_row(const LogProbsArgs &p, int64_t row, const Sums &x, uint64_t list, int lane)
{
    const bool empty = x.s == 0.0f;   // the largest logit adds about 1, so: nothing but -infinity
    const float none = -__builtin_inff();
    const float log_s = logf(x.s);    // -infinity of 0
    const float a = p.scale * kLog2e;
    const float total = __builtin_fmaf(-kLn2, lacking(x.m, a), log_s);
    if (lane == 0) {
        if (p.tokens != nullptr) {
            const int t = p.tokens[row];
            float lp = 0.0f;
            if (t >= 0 && t < p.vocab)
                lp = empty ? none : p.scale * (logit_at<BF16>(p.logits, row * p.ld + t) - x.m) - total;
            p.logprob[row] = lp;
        }
        if (p.entropy != nullptr) p.entropy[row] = empty ? 0.0f : log_s - kLn2 * (x.u / x.s);
        if (p.stats != nullptr) {
            p.stats[2 * row] = empty ? none : x.s != x.s ? x.s : x.m;
            p.stats[2 * row + 1] = total;
        }
    }
    if (lane < p.top) {
        p.top_ids[row * p.top + lane] = place_of(list);
        if (p.top_logprobs != nullptr)
            p.top_logprobs[row * p.top + lane] =
                empty ? none : p.scale * (value_of((uint32_t)(list >> 32)) - x.m) - total;
    }
}

// One row's chunk in registers: 32 logits per lane, in 16-byte vectors.  Vectors
// lie at 16-byte boundaries whatever the row's address: the first and the last may
// hold values of other rows or none (16 bytes that hold one value of the row lie on
// its page), which are masked.
template <bool BF16>
struct Chunk {
    static constexpr int VEC = BF16 ? 8 : 4, U = 32 / VEC;
    u32x4 v[U];

    __device__ __forceinline__ void load(const unsigned char *row16, int64_t chunk, int vectors, int lane)
    {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t at = (chunk * U + i) * 64 + lane;
            v[i] = load16(row16 + 16 * (at < vectors ? at : vectors - 1));
        }
    }
    __device__ __forceinline__ float operator[](int j) const
    {
        const uint32_t w = v[j / VEC][BF16 ? j % VEC / 2 : j % VEC];
        return __uint_as_float(!BF16 ? w : j & 1 ? w & 0xFFFF0000u : w << 16);
    }
};

template <bool BF16, bool TOP>
__global__ void __launch_bounds__(256) log_probs_kernel(LogProbsArgs p)
{
    using C = Chunk<BF16>;
    constexpr int ES = BF16 ? 2 : 4;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int member = p.team == 1 ? 0 : wave;
    const int64_t units = p.rows * p.parts;
    const float a = p.scale * kLog2e;
    __shared__ float team_sums[4][3];
    __shared__ uint64_t team_lists[4][64];
    __shared__ __attribute__((aligned(16))) float spread[4][32];

    for (int64_t unit0 = (int64_t)blockIdx.x * (4 / p.team); unit0 < units; unit0 += (int64_t)gridDim.x * (4 / p.team)) {
        const int64_t unit = unit0 + (p.team == 1 ? wave : 0);
        if (unit >= units) break;   // of single waves only: teams leave together
        const int64_t row = unit / p.parts;
        const int part = (int)(unit - row * p.parts);
        const uintptr_t start = (uintptr_t)p.logits + (uintptr_t)(row * p.ld) * ES;
        const int head = (int)(start & 15) / ES;    // values before the row in its first vector
        const unsigned char *row16 = reinterpret_cast<const unsigned char *>(start & ~(uintptr_t)15);
        const int vectors = (int)(((int64_t)head + p.vocab + C::VEC - 1) / C::VEC);
        const int chunks = (vectors + 64 * C::U - 1) / (64 * C::U);
        const int begin = part * p.part_chunks, end = min(chunks, begin + p.part_chunks);

        Sums x;
        TopList top(lane, p.top);
        float bar = __builtin_nanf("");   // the list's last value; NaN while it is not full
        C cur, nxt;
        int c = begin + member;
        if (c < end) cur.load(row16, c, vectors, lane);
        for (; c < end; c += p.team) {
            if (c + p.team < end) nxt.load(row16, c + p.team, vectors, lane);
            // place of this lane's first value; value j lies 64 VEC further per vector
            const int first = (c * C::U * 64 + lane) * C::VEC - head;
            auto place = [](int first, int j) { return first + j / C::VEC * (64 * C::VEC) + j % C::VEC; };
            const bool whole = c * CHUNK >= head && (c + 1) * CHUNK - head <= p.vocab;
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = cur[j];
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if ((unsigned)place(first, j) >= (unsigned)p.vocab) z[j] = -__builtin_inff();
            }
            float largest = z[0];
#pragma unroll
            for (int j = 1; j < 32; ++j) largest = fmaxf(largest, z[j]);
            // Later chunks have higher places, so a value has to exceed the last one's.
            if (TOP && __ballot(!(largest <= bar)) != 0) {
                top.template absorb_values<32>(z, largest, p.vocab, first, place, spread[wave]);
                if (top.least != 0) bar = value_of((uint32_t)(top.least >> 32));
            }
            x.move(fmaxf(x.m, largest), a);
            float s[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
            auto terms = [&](auto exponent) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float t = exponent(z[j]), e = __builtin_amdgcn_exp2f(t);
                    s[j & 3] += e;
                    u[j & 3] = __builtin_fmaf(e, bounded(t), u[j & 3]);
                }
            };
            const float c_m = a * x.m;
            if (__ballot(huge(x.m, a)) == 0) {
                terms([&](float v) { return __builtin_fmaf(a, v, -c_m); });
            } else {
                const float rest = lacking(x.m, a);
                terms([&](float v) { return a * (v - x.m) + rest; });
            }
            x.s += (s[0] + s[1]) + (s[2] + s[3]);
            x.u += (u[0] + u[1]) + (u[2] + u[3]);
            cur = nxt;
        }
        x.add_lanes(a);
        uint64_t list = top.list;
        if (p.team > 1) {
            if (lane == 0) {
                team_sums[wave][0] = x.m;
                team_sums[wave][1] = x.s;
                team_sums[wave][2] = x.u;
            }
            if (TOP) team_lists[wave][lane] = list;
            __syncthreads();
            if (TOP && wave < 2) {
                list = merged(list, team_lists[wave + 2][lane]);
                if (wave == 1) team_lists[1][lane] = list;
            }
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int w = 1; w < 4; ++w) x.add(Sums{team_sums[w][0], team_sums[w][1], team_sums[w][2]}, a);
                if (TOP) list = merged(list, team_lists[1][lane]);
            }
            __syncthreads();
            if (wave != 0) continue;
        }
        if (p.parts == 1) {
            finish_row<BF16>(p, row, x, list, lane);
        } else {
            if (lane == 0) *reinterpret_cast<floatx4 *>(p.ws + 4 * unit) = floatx4{x.m, x.s, x.u, 0.0f};
            if (TOP && lane < p.top) p.ws_keys[unit * p.top + lane] = list;
        }
    }
}

// The parts of a row: four waves take every fourth list each and merge them (they
// are sorted), then their own.
template <bool BF16>
__global__ void __launch_bounds__(256) log_probs_join_kernel(LogProbsArgs p)
{
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const float a = p.scale * kLog2e;
    __shared__ uint64_t lists[4][64];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const uint64_t *keys = p.ws_keys + row * p.parts * p.top;
        uint64_t list = 0;
        if (p.top > 0) {
            auto part = [&](int i) { return i < p.parts && lane < p.top ? keys[i * p.top + lane] : 0; };
            list = part(wave);
            uint64_t next = part(wave + 4);
            for (int i = wave + 4; i < p.parts; i += 4) {
                const uint64_t k = next;
                next = part(i + 4);
                list = merged(list, k);
            }
            lists[wave][lane] = list;
        }
        Sums x;
        if (wave == 0) {
            for (int i = lane; i < p.parts; i += 64) {
                const floatx4 v = *reinterpret_cast<const floatx4 *>(p.ws + 4 * (row * p.parts + i));
                x.add(Sums{v[0], v[1], v[2]}, a);
            }
            x.add_lanes(a);
        }
        __syncthreads();
        if (wave == 0) {
            if (p.top > 0)
#pragma nounroll
                for (int w = 1; w < 4; ++w) list = merged(list, lists[w][lane]);
            finish_row<BF16>(p, row, x, list, lane);
        }
        __syncthreads();
    }
}

// --------------------------------------------------------------- gradient --
//
//     dz_j = p_j (c + b t_j) [+ scale g at the token],   t_j = log2 p_j,  p_j = 2^t_j
//     c = -scale (g + h entropy),   b = -scale h ln2
//
// Bound by HBM: one read and one write of the logits (4096 x 32768 bf16, 537 MB: 85 us,
// 6.3 TB/s, part of it from the memory-side cache).  A wave takes 64 * U vectors of a row.
template <bool BF16>
__global__ void __launch_bounds__(256) log_probs_grad_kernel(LogProbsGradArgs p, int segments)
{
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES, U = 4;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t units = p.rows * segments;
    const float a = p.scale * kLog2e;
    for (int64_t unit = (int64_t)blockIdx.x * 4 + wave; unit < units; unit += (int64_t)gridDim.x * 4) {
        const int64_t row = unit / segments;
        const int segment = (int)(unit - row * segments);
        const uintptr_t start = (uintptr_t)p.logits + (uintptr_t)(row * p.ld) * ES;
        unsigned char *out = static_cast<unsigned char *>(p.dlogits) + row * p.ldd * ES;
        // vectors at 16-byte boundaries of the logits, as in Chunk
        const int head = (int)(start & 15) / ES;
        const unsigned char *row16 = reinterpret_cast<const unsigned char *>(start & ~(uintptr_t)15);
        const int vectors = (int)(((int64_t)head + p.vocab + VEC - 1) / VEC);
        const bool same = (((uintptr_t)out ^ start) & 15) == 0;   // the outputs' boundaries are the logits'

        int token = p.dlogprob != nullptr ? p.tokens[row] : -1;
        if (token >= p.vocab) token = -1;
        const float g = token >= 0 ? p.dlogprob[row] : 0.0f;
        const float h = p.dentropy != nullptr ? p.dentropy[row] : 0.0f;
        const float m = p.stats[2 * row], total = p.stats[2 * row + 1];
        const bool zero = (g == 0.0f && h == 0.0f) || m == -__builtin_inff();
        const float c = -p.scale * (h != 0.0f ? __builtin_fmaf(h, p.entropy[row], g) : g), b = -p.scale * h * kLn2;
        const float shift = total * kLog2e, extra = p.scale * g;

        const int64_t v0 = (int64_t)segment * (64 * U) + lane;
        u32x4 w[U];
        if (!zero) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t at = v0 + 64 * i;
                w[i] = load16(row16 + 16 * (at < vectors ? at : vectors - 1));
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (v0 + 64 * i >= vectors) break;
            const int first = (int)((v0 + 64 * i) * VEC) - head;   // place of the vector's first value
            float d[VEC];
            if (zero) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) d[j] = 0.0f;
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float z = BF16 ? __uint_as_float(j & 1 ? w[i][j / 2] & 0xFFFF0000u : w[i][j / 2] << 16)
                                         : __uint_as_float(w[i][j & 3]);
                    const float t = __builtin_fmaf(a, z - m, -shift);
                    d[j] = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(b, bounded(t), c);
                }
                if (token >= first && token < first + VEC) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) d[j] += token == first + j ? extra : 0.0f;
                }
            }
            if (same && first >= 0 && first + VEC <= p.vocab) {
                u32x4 r;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r[j] = BF16 ? f32x2_to_bf16x2_rne(d[(2 * j) % VEC], d[(2 * j + 1) % VEC]) : __float_as_uint(d[j]);
                __builtin_nontemporal_store(r, reinterpret_cast<u32x4 *>(out + (int64_t)first * ES));
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (first + j < 0 || first + j >= p.vocab) continue;
                    if (BF16)
                        reinterpret_cast<uint16_t *>(out)[first + j] = f32_to_bf16_rne(d[j]);
                    else
                        reinterpret_cast<float *>(out)[first + j] = d[j];
                }
            }
        }
    }
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20); }   // loops cover the rest

}  // namespace

int log_probs_chunk() { return CHUNK; }

hipError_t launch_log_probs(const LogProbsArgs &a, bool bf16, hipStream_t stream)
{
    const int per = 4 / a.team;
    const unsigned grid = grid_of((a.rows * a.parts + per - 1) / per);
    auto kernel = bf16 ? (a.top > 0 ? log_probs_kernel<true, true> : log_probs_kernel<true, false>)
                       : (a.top > 0 ? log_probs_kernel<false, true> : log_probs_kernel<false, false>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.parts == 1) return err;
    auto join = bf16 ? log_probs_join_kernel<true> : log_probs_join_kernel<false>;
    hipLaunchKernelGGL(join, dim3(grid_of(a.rows)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_log_probs_grad(const LogProbsGradArgs &a, bool bf16, hipStream_t stream)
{
    const int vec = bf16 ? 8 : 4;
    // vectors of a row, one more where its first value is not at a boundary
    const int64_t vectors = ((int64_t)a.vocab + 2 * (vec - 1)) / vec;
    const int segments = (int)((vectors + 255) / 256);
    const unsigned grid = grid_of((a.rows * segments + 3) / 4);
    auto kernel = bf16 ? log_probs_grad_kernel<true> : log_probs_grad_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, a, segments);
    return hipGetLastError();
}

}  // namespace dg
