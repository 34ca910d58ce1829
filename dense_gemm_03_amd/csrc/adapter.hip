// The first of the adapters' two products: t = scale x . a^T, each row with the a of
// its own adapter.
//
// A block has 64 rows, of which a product takes those of one adapter at a time, and a
// part of K.  Few blocks stream slowly (a compute unit takes 25 KB per us), so parts
// spread the adapters' bytes; t of a few rows is left as the parts' sums, others' are
// joined (5 us).  1 row, rank 16, K = 4096: 5.9 us; 4096 rows of 8 requests: 16 us, with
// rank 64 25 us, most of it reads of a through L2, once per 64 rows.  Rows in blocks of 16,
// sixteen waves and one part took 8 us for one row, 20 and 44 us for 4096.
#include "serving.hpp"
#include "strip.hpp"

namespace dg {
namespace {

constexpr int WV = 8;

// A value of t as the product reads it.
template <bool BF16>
__device__ __forceinline__ void store_t(const AdapterDownArgs &p, int64_t at, float v)
{
    if constexpr (BF16) {
        uint16_t *t = static_cast<uint16_t *>(p.t);
        const uint16_t hi = f32_to_bf16_rne(v);
        const float rest = v - __uint_as_float((uint32_t)hi << 16);
        t[at] = hi;
        t[p.plane + at] = f32_to_bf16_rne(fabsf(rest) < __builtin_inff() ? rest : 0.0f);   // infinity has none
    } else {
        static_cast<float *>(p.t)[at] = v;
    }
}

template <bool BF16, int W>
__global__ void __launch_bounds__(64 * WV) adapter_down_kernel(AdapterDownArgs p)
{
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ int list[64];
    __shared__ float sums[WV / 2 * 64 * 16 * W];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int groups = (p.rows + 63) / 64, at = (int)blockIdx.x / p.parts;
    const int part = (int)blockIdx.x % p.parts, row0 = at % groups * 64, slot = at / groups;
    const int k0 = part * p.part_k, len = min(p.part_k, p.K - k0);

    int id = row0 + lane < p.rows ? p.ids[row0 + lane] : -1;
    if ((unsigned)id >= (unsigned)p.count) id = -1;
    int turn = 0;
    for (uint64_t left = __ballot(id >= 0); left != 0; turn = turn + 1 == p.slots ? 0 : turn + 1) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(id == e);
        left &= ~mine;
        if (turn != slot) continue;
        if (wave == 0 && id == e) list[lanes_below(mine)] = row0 + lane;
        __syncthreads();
        const int count = __builtin_popcountll(mine);
        const float scale = p.scales != nullptr ? p.scales[e] : 1.0f;
        const In *a = static_cast<const In *>(p.a) + e * p.stride_a + k0;
        for (int n0 = 0; n0 < p.rank; n0 += 16 * W) {
            auto tile = [&](auto rt_c, auto u_c) {
                product<WV, BF16, true, W, 1, 1, decltype(rt_c)::value, decltype(u_c)::value>(
                    a, p.lda, p.rank, len, n0, p.x, 0, count,
                    [&](int r) { return (int64_t)list[r] * p.ldx + k0; }, sums, lane, wave,
                    [&](int r, int col, const float (&z)[1]) {
                        const int64_t to = (int64_t)list[r] * p.pitch + n0 + col;
                        if (p.parts > 1)
                            p.ws[(int64_t)part * p.rows * p.pitch + to] = scale * z[0];
                        else
                            store_t<BF16>(p, to, scale * z[0]);
                    });
            };
            using std::integral_constant;
            if (count <= 16)
                tile(integral_constant<int, 1>(), integral_constant<int, W == 4 ? 2 : 4>());
            else if (count <= 32)
                tile(integral_constant<int, 2>(), integral_constant<int, 2>());
            else
                tile(integral_constant<int, 4>(), integral_constant<int, 2>());
            __syncthreads();   // the sums and the list are read
        }
    }
}

// t from the sums of parts.
template <bool BF16>
__global__ void __launch_bounds__(256) adapter_join_kernel(AdapterDownArgs p)
{
    const int64_t total = (int64_t)p.rows * p.rank;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / p.rank, at = row * p.pitch + (i - row * p.rank);
        const int e = p.ids[row];
        if ((unsigned)e >= (unsigned)p.count) continue;
        float v[ADAPTER_MAX_PARTS];
#pragma unroll
        for (int z = 0; z < ADAPTER_MAX_PARTS; ++z) v[z] = z < p.parts ? p.ws[(int64_t)z * p.rows * p.pitch + at] : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int z = 0; z < ADAPTER_MAX_PARTS; ++z) sum += v[z];
        store_t<BF16>(p, at, sum);
    }
}

// K below 8, which the vectors above do not fit: a thread per value.
template <bool BF16>
__global__ void __launch_bounds__(256) adapter_small_kernel(AdapterDownArgs p)
{
    const int64_t total = (int64_t)p.rows * p.rank;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / p.rank;
        const int r = (int)(i - row * p.rank), e = p.ids[row];
        if ((unsigned)e >= (unsigned)p.count) continue;
        float z = 0.0f;
        for (int k = 0; k < p.K; ++k) {
            if (BF16)
                z += __uint_as_float((uint32_t) static_cast<const uint16_t *>(p.x)[row * p.ldx + k] << 16) *
                     __uint_as_float((uint32_t) static_cast<const uint16_t *>(p.a)[e * p.stride_a + r * p.lda + k] << 16);
            else
                z += static_cast<const float *>(p.x)[row * p.ldx + k] *
                     static_cast<const float *>(p.a)[e * p.stride_a + r * p.lda + k];
        }
        store_t<BF16>(p, row * p.pitch + r, (p.scales != nullptr ? p.scales[e] : 1.0f) * z);
    }
}

}  // namespace

hipError_t launch_adapter_down(const AdapterDownArgs &a, bool bf16, hipStream_t stream)
{
    const int64_t values = ((int64_t)a.rows * a.rank + 255) / 256;
    const dim3 flat((unsigned)(values < 65536 ? values : 65536));
    if (a.K < 8) {
        hipLaunchKernelGGL((bf16 ? adapter_small_kernel<true> : adapter_small_kernel<false>), flat, dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    }
    // ranks in strips of 16, 32 or 64
    auto kernel = bf16 ? (a.rank <= 16   ? adapter_down_kernel<true, 1>
                          : a.rank <= 32 ? adapter_down_kernel<true, 2>
                                         : adapter_down_kernel<true, 4>)
                       : (a.rank <= 16   ? adapter_down_kernel<false, 1>
                          : a.rank <= 32 ? adapter_down_kernel<false, 2>
                                         : adapter_down_kernel<false, 4>);
    const int64_t blocks = (int64_t)((a.rows + 63) / 64) * a.slots * a.parts;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * WV), 0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || a.parts == 1 || !a.join) return err;
    hipLaunchKernelGGL((bf16 ? adapter_join_kernel<true> : adapter_join_kernel<false>), flat, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dg
