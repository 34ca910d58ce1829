// The first of the adapters' two products: t = scale x . a^T, each row with the a of
// its own adapter.
//
// A block has 64 rows and goes through their adapters (the slots-th of them each), for
// the rows that have it, over its part of K.  Bound by the adapters' bytes when there
// are few rows; with long prompts by the L2 reads of a, once per 64 rows.
#include "serving.hpp"
#include "strip.hpp"

namespace dg {
namespace {

constexpr int WV = 8;

template <bool BF16, int W>
__global__ void __launch_bounds__(64 * WV) adapter_down_kernel(AdapterDownArgs p)
{
    using In = typename std::conditional<BF16, uint16_t, float>::type;
    __shared__ int list[64];
    __shared__ float sums[WV / 2 * 64 * 16 * W];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = (int)blockIdx.x % p.slots, rest = (int)blockIdx.x / p.slots;
    const int part = rest % p.parts, row0 = rest / p.parts * 64;
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
        float *t = p.t + part * p.t_part;
        for (int n0 = 0; n0 < p.rank; n0 += 16 * W) {
            auto tile = [&](auto rt_c, auto u_c) {
                product<WV, BF16, true, W, 1, 1, decltype(rt_c)::value, decltype(u_c)::value>(
                    a, p.lda, p.rank, len, n0, p.x, 0, count,
                    [&](int r) { return (int64_t)list[r] * p.ldx + k0; }, sums, lane, wave,
                    [&](int r, int col, const float (&z)[1]) { t[(int64_t)list[r] * p.pitch + n0 + col] = scale * z[0]; });
            };
            using std::integral_constant;
            if (count <= 16)
                tile(integral_constant<int, 1>(), integral_constant<int, 2>());
            else if (count <= 32)
                tile(integral_constant<int, 2>(), integral_constant<int, 2>());
            else
                tile(integral_constant<int, 4>(), integral_constant<int, 2>());
            __syncthreads();   // the sums and the list are read
        }
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
        p.t[row * p.pitch + r] = (p.scales != nullptr ? p.scales[e] : 1.0f) * z;
    }
}

}  // namespace

hipError_t launch_adapter_down(const AdapterDownArgs &a, bool bf16, hipStream_t stream)
{
    if (a.K < 8) {
        const int64_t blocks = ((int64_t)a.rows * a.rank + 255) / 256;
        hipLaunchKernelGGL((bf16 ? adapter_small_kernel<true> : adapter_small_kernel<false>),
                           dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream, a);
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
    return hipGetLastError();
}

}  // namespace dg
