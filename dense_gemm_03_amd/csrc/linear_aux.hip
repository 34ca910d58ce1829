// The linear layers' kernel table and the kernels next to the products: the
// reduce of partial sums, and the gradient through the epilogue (dz, dbias).
#include "linear_configs.hpp"

namespace dg {

const LinearConfig *linear_configs(int dtype, int *count)
{
    static const LinearConfig f32[] = {DG_LIN_F32_TABLE(DG_LIN_ENTRY) DG_LIN_F32_ROWS(DG_LIN_ROWS_ENTRY)};
    static const LinearConfig bf16[] = {DG_LIN_BF16_TABLE(DG_LIN_ENTRY) DG_LIN_BF16_ROWS(DG_LIN_ROWS_ENTRY)};
    *count = dtype == 0 ? (int)(sizeof(f32) / sizeof(f32[0])) : (int)(sizeof(bf16) / sizeof(bf16[0]));
    return dtype == 0 ? f32 : bf16;
}

namespace {

// Group of `row` (lo <= row < hi of exactly one group), or -1 outside all.
__device__ __forceinline__ int group_of_row(const int32_t *offsets, int groups, int rows, int row)
{
    int a = 0, b = groups;   // the last g in [a, b) with offsets[g] <= row
    if (row < clamp_row(offsets[0], rows) || row >= clamp_row(offsets[groups], rows)) return -1;
    while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (clamp_row(offsets[mid], rows) <= row)
            a = mid;
        else
            b = mid;
    }
    return a;
}

// One thread finishes pieces of V consecutive columns: the slices' sums in
// slice order, then the epilogue of the product kernels.
template <int V, bool WGRAD>
__global__ void __launch_bounds__(256) linear_reduce_kernel(LinearArgs p)
{
    const int pieces = (p.N + V - 1) / V;
    const int64_t out_rows = WGRAD ? (int64_t)p.groups * p.M : p.rows;
    const int64_t total = out_rows * pieces, slice = out_rows * p.N;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < total; id += (int64_t)gridDim.x * 256) {
        const int64_t row = id / pieces;
        const int col = (int)(id - row * pieces) * V, n = p.N - col;
        int group = 0;
        if (WGRAD)
            group = (int)(row / p.M);
        else if (p.offsets != nullptr && (group = group_of_row(p.offsets, p.groups, p.rows, (int)row)) < 0)
            continue;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
        const float *w = p.ws + row * p.N + col;
        if (V > 1 && (p.N & 3) == 0) {
#pragma unroll 4
            for (int z = 0; z < p.splits; ++z)
#pragma unroll
                for (int h = 0; h < V; h += 4)
                    if (h < n) {
                        const u32x4 q = load16(w + z * slice + h);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[(h + i) & (V - 1)] += __uint_as_float(q[i]);
                    }
        } else {
#pragma unroll 4
            for (int z = 0; z < p.splits; ++z)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < n) v[i] += w[z * slice + i];
        }
        float bias[V];
        load_bias<V>(p.e, group * p.stride_bias + col, n, bias);
        finish_piece<V>(p.e, WGRAD ? group * p.stride_c : 0, WGRAD ? row - (int64_t)group * p.M : row,
                        col, n, bias, v);
    }
}

// dz = dy act'(pre), and each column's sum over the block's rows.  A block
// takes 64 V columns of one chunk of rows of one group, or (CHUNKS false) of a
// whole group, whose sums are then the result; its WV waves walk the rows in
// turn, V columns per lane, and the sums meet in LDS.  dz is rounded to the
// operands' type, once: the matrix cores multiply bf16 with bf16 only, and dz as
// two bf16 terms would double both products.  The sums take it unrounded.
// Bound by HBM: 2 reads and 1 write of rows x N.  16-byte rows are taken 16
// bytes per lane (1 KiB of a row per wave), others with the lanes side by side,
// element by element.  V == 1 spreads few columns over more blocks.
template <bool BF16, int V, bool CHUNKS>
__global__ void __launch_bounds__(CHUNKS ? 256 : 1024) act_grad_kernel(ActGradArgs p, int col_blocks)
{
    constexpr bool WIDE = V > 1;
    constexpr int WV = CHUNKS ? 4 : 16;
    __shared__ float sums[WV][64 * V];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int tile = (int)blockIdx.x / col_blocks, cb = (int)blockIdx.x - tile * col_blocks;
    int lo, first = 0, count;
    if constexpr (CHUNKS) {
        const GroupRows list(p.offsets, p.groups, p.rows, p.chunk_rows, lane);
        if (tile >= list.total) return;
        int group, m, tm;
        list.find(p.offsets, p.groups, p.rows, p.chunk_rows, lane, 0, false, tile, group, lo, m, tm);
        first = tm * p.chunk_rows;
        count = min(p.chunk_rows, m - first);
    } else {
        group_span(p.offsets, tile, p.rows, lo, count);
    }
    const int col0 = cb * 64 * V, last = p.N - 1 - col0;
    // lane's columns: V in a row, or every 64th
    const bool vec = WIDE && p.vec != 0;
    auto column = [&](int i) { return vec ? lane * V + i : lane + 64 * i; };
    auto load = [&](const void *X, int64_t at, bool bf16, float (&v)[V]) {
        if (vec && bf16 == BF16 && p.N - col0 - lane * V >= V) {
            load_out<V, WIDE>(X, at + lane * V, V, BF16, true, v);
        } else if (bf16) {
            // past the edge the last column's value, which nothing takes up: no
            // branch, so that the loads are under way together
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = __uint_as_float((uint32_t) static_cast<const uint16_t *>(X)[at + min(column(i), last)] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = static_cast<const float *>(X)[at + min(column(i), last)];
        }
    };
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 0.0f;
#pragma unroll 4
    for (int r = wave; r < count; r += WV) {
        const int64_t row = lo + first + r;
        float g[V], z[V];
        load(p.dy, row * p.lddy + col0, BF16, g);
        if (p.act != ACT_NONE) {
            load(p.pre, row * p.ldp + col0, p.pre_bf16 != 0, z);
            act_slope<V, !BF16>(p.act, z);
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] *= z[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] += col0 + column(i) < p.N ? g[i] : 0.0f;
        if (p.dz == nullptr) continue;
        const int64_t at = row * p.lddz + col0;
        if (vec && p.N - col0 - lane * V >= V) {
            store_outs<V, WIDE>(p.dz, at + lane * V, V, BF16, true, g);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (col0 + column(i) >= p.N) continue;
                if (BF16)
                    static_cast<uint16_t *>(p.dz)[at + column(i)] = f32_to_bf16_rne(g[i]);
                else
                    static_cast<float *>(p.dz)[at + column(i)] = g[i];
            }
        }
    }
    if (p.dbias == nullptr) return;
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][column(i)] = s[i];
    __syncthreads();
    float *out = (CHUNKS ? p.ws : p.dbias) + (int64_t)tile * p.N;
    for (int i = (int)threadIdx.x; i < 64 * V; i += 64 * WV)
        if (col0 + i < p.N) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < WV; ++w) t += sums[w][i];
            out[col0 + i] = t;
        }
}

// dbias of one group: its chunks' sums (none: zero).  Four threads per column
// take every fourth chunk each, in order.
__global__ void __launch_bounds__(256) bias_reduce_kernel(ActGradArgs p, int col_blocks)
{
    __shared__ float sums[4][64];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int group = (int)blockIdx.x / col_blocks, cb = (int)blockIdx.x - group * col_blocks;
    int first = 0, mine = 0;   // the group's first chunk, and its chunks
    if (p.offsets == nullptr) {
        mine = (p.rows + p.chunk_rows - 1) / p.chunk_rows;
    } else {
        for (int base = 0; base <= group; base += 64) {
            int lo, m;
            const int t = GroupRows::lane_tiles(p.offsets, base + lane, p.groups, p.rows, p.chunk_rows, 0,
                                                false, lo, m);
            const int upto = GroupRows::scan(t, lane);
            const int at = min(63, group - base);   // the group itself, or the last of these 64
            first = min(first + __builtin_amdgcn_readlane(upto, at), GroupRows::CAP);
            mine = __builtin_amdgcn_readlane(t, at);
        }
        first -= mine;
        // offsets that fall can give rows to several groups, and more chunks
        // than there is room for
        first = min(first, p.chunks);
        mine = min(mine, p.chunks - first);
    }
    const int j = cb * 64 + lane;
    const float *w = p.ws + (int64_t)first * p.N + j;
    float s = 0.0f;
    if (j < p.N) {
#pragma unroll 8
        for (int t = wave; t < mine; t += 4) s += w[(int64_t)t * p.N];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && j < p.N)
        p.dbias[(int64_t)group * p.N + j] = sums[0][lane] + sums[1][lane] + sums[2][lane] + sums[3][lane];
}

unsigned grid_of(int64_t work)
{
    const int64_t blocks = (work + 255) / 256;
    return (unsigned)(blocks < 1 ? 1 : blocks > 65536 ? 65536 : blocks);   // the loop covers the rest
}

}  // namespace

hipError_t launch_linear_reduce(const LinearArgs &a, bool weight_grad, hipStream_t stream)
{
    const int64_t rows = weight_grad ? (int64_t)a.groups * a.M : a.rows;
    // 16 bytes of output per thread; fewer where that leaves most of the chip
    // without a thread, one value where rows have no 16-byte alignment
    const int64_t all = rows * a.N;
    const int V = all <= 65536 || !a.e.vec || a.N % 4 != 0 ? 1 : a.e.out_bf16 && all > (1 << 21) ? 8 : 4;
    const dim3 grid(grid_of(rows * ((a.N + V - 1) / V)));
    auto kernel = weight_grad ? (V == 8   ? linear_reduce_kernel<8, true>
                                 : V == 4 ? linear_reduce_kernel<4, true>
                                          : linear_reduce_kernel<1, true>)
                              : (V == 8   ? linear_reduce_kernel<8, false>
                                 : V == 4 ? linear_reduce_kernel<4, false>
                                          : linear_reduce_kernel<1, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t stream)
{
    const int W = a.bf16 ? 8 : 4;
    const bool whole = a.chunk_rows == 0;
    const int parts = whole ? a.groups : a.chunks;
    // 16 bytes per lane, unless that leaves most of the chip idle; rows that are
    // taken element by element want more waves (777 x 1025 fp32: 10.4 us in 245
    // blocks, 7.4 in 833)
    const bool wide = (int64_t)parts * ((a.N + 64 * W - 1) / (64 * W)) >= (a.vec ? 64 : 1024);
    const int V = wide ? W : 1;
    const int col_blocks = (a.N + 64 * V - 1) / (64 * V);
    if (parts > 0) {
        auto kernel = a.bf16 ? (whole ? (wide ? act_grad_kernel<true, 8, false> : act_grad_kernel<true, 1, false>)
                                      : (wide ? act_grad_kernel<true, 8, true> : act_grad_kernel<true, 1, true>))
                             : (whole ? (wide ? act_grad_kernel<false, 4, false> : act_grad_kernel<false, 1, false>)
                                      : (wide ? act_grad_kernel<false, 4, true> : act_grad_kernel<false, 1, true>));
        hipLaunchKernelGGL(kernel, dim3((unsigned)(parts * col_blocks)), dim3(whole ? 1024 : 256), 0, stream, a,
                           col_blocks);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    if (a.dbias != nullptr && !whole) {
        const int cb = (a.N + 63) / 64;
        hipLaunchKernelGGL(bias_reduce_kernel, dim3((unsigned)(cb * a.groups)), dim3(256), 0, stream, a, cb);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace dg
