// Kernel table of the linear layers: one entry per tile shape, with launchers
// for y = x . w (w as K x N, or as N x K) and for dw = x^T . dz, each for
// 16-byte aligned rows and for any alignment of the element type.
//
//   X(NAME, BF16, BM, BN, BK, WM, WN, STAGES, GROUP_M, STEP, ALONE, BLOCK)
//
// The last three are times in us that the dispatcher ranks the entries by
// (linear_api.hip): of a k-tile per block on a full compute unit, of a k-tile
// of a block that has the unit to itself, and of a block's start and end.
#pragma once

#include <hip/hip_runtime.h>

#include "linear_kernel.hpp"

namespace dg {

typedef hipError_t (*linear_fn)(const LinearArgs &args, int blocks, hipStream_t stream);

template <bool BF16, int FORM, int W, int WV>
hipError_t launch_few_rows(const LinearArgs &args, int blocks, hipStream_t stream);

enum { FORM_N = 0, FORM_T = 1, FORM_WGRAD = 2 };

struct LinearConfig {
    const char *name;
    float step, alone, block;
    int bm, bn, bk, threads, stages, group_m;   // stages == 0: the kernel for few rows
    linear_fn fn[3][2];   // by form; [0] aligned, [1] not; nullptr where there is none
};

template <bool BF16, int BM, int BN, int BK, int WM, int WN, int STAGES, int LX, int LW, bool ALIGNED>
hipError_t launch_linear(const LinearArgs &args, int blocks, hipStream_t stream);

// how x and w (dz) lie in memory
#define DG_LIN_LX_N ::dg::KMAJOR
#define DG_LIN_LW_N ::dg::MNMAJOR
#define DG_LIN_LX_T ::dg::KMAJOR
#define DG_LIN_LW_T ::dg::KMAJOR
#define DG_LIN_LX_W ::dg::MNMAJOR
#define DG_LIN_LW_W ::dg::MNMAJOR

#define DG_LIN_F32_TABLE(X)                                                                  \
    X("f32_256x256x32_w4x2_s2", false, 256, 256, 32, 4, 2, 2, 8, 7.03f, 0.8f, 6.0f)          \
    X("f32_128x128x32_w2x2_s2", false, 128, 128, 32, 2, 2, 2, 8, 1.87f, 1.2f, 4.0f)          \
    X("f32_64x64x32_w2x2_s3", false, 64, 64, 32, 2, 2, 3, 8, 0.48f, 0.51f, 0.83f)

// Small bf16 tiles have three or four stages: two leave less than a k-tile's
// products to cover a load, and where a unit has one block every k-tile waits
// (0.44 us per k-tile of 64 x 64 with two stages, 0.20 with four).  With two,
// five blocks share a unit, which is better than three stages where a block has a
// k-tile or two and its stores are what counts (12 groups of about one row, 1088 x
// 4864, the backward pass: 80 us against 92).
#define DG_LIN_BF16_TABLE(X)                                                                 \
    X("bf16_256x256x64_w2x2_s2", true, 256, 256, 64, 2, 2, 2, 8, 1.45f, 0.60f, 6.6f)         \
    X("bf16_128x128x64_w2x2_s2", true, 128, 128, 64, 2, 2, 2, 8, 0.45f, 0.565f, 1.1f)        \
    X("bf16_64x128x64_w1x4_s3", true, 64, 128, 64, 1, 4, 3, 8, 0.32f, 0.33f, 0.75f)          \
    X("bf16_64x64x64_w2x2_s2", true, 64, 64, 64, 2, 2, 2, 8, 0.20f, 0.42f, 0.05f)            \
    X("bf16_64x64x64_w2x2_s4", true, 64, 64, 64, 2, 2, 4, 8, 0.21f, 0.215f, 0.3f)

// Entries for few rows: X(NAME, BF16, FORM (N or T), W, waves); 16 rows, 16 W columns.
#define DG_LIN_F32_ROWS(X)                       \
    X("f32_rows_n_w2x8", false, N, 2, 8)         \
    X("f32_rows_n_w4x8", false, N, 4, 8)         \
    X("f32_rows_t_w1x8", false, T, 1, 8)         \
    X("f32_rows_t_w2x8", false, T, 2, 8)

#define DG_LIN_BF16_ROWS(X)                      \
    X("bf16_rows_n_w2x8", true, N, 2, 8)         \
    X("bf16_rows_n_w4x8", true, N, 4, 8)         \
    X("bf16_rows_t_w1x8", true, T, 1, 8)         \
    X("bf16_rows_t_w2x8", true, T, 2, 8)

#define DG_LIN_FORM_ID_N 0
#define DG_LIN_FORM_ID_T 1
#define DG_LIN_ROWS_FN(BF16, F, W, WV)                     \
    {&launch_few_rows<BF16, DG_LIN_FORM_ID_##F, W, WV>,    \
     &launch_few_rows<BF16, DG_LIN_FORM_ID_##F, W, WV>}
#define DG_LIN_ROWS_FNS_N(...) {DG_LIN_ROWS_FN(__VA_ARGS__), DG_LIN_NOFNS, DG_LIN_NOFNS}
#define DG_LIN_ROWS_FNS_T(...) {DG_LIN_NOFNS, DG_LIN_ROWS_FN(__VA_ARGS__), DG_LIN_NOFNS}
#define DG_LIN_ROWS_ENTRY(NAME, BF16, F, W, WV) \
    LinearConfig{NAME, 0, 0, 0, 16, 16 * (W), 1, 64 * (WV), 0, 1, DG_LIN_ROWS_FNS_##F(BF16, F, W, WV)},

#define DG_LIN_FNS(BF16, BM, BN, BK, WM, WN, S, F)                                              \
    {&launch_linear<BF16, BM, BN, BK, WM, WN, S, DG_LIN_LX_##F, DG_LIN_LW_##F, true>,           \
     &launch_linear<BF16, BM, BN, BK, WM, WN, S, DG_LIN_LX_##F, DG_LIN_LW_##F, false>}
#define DG_LIN_NOFNS {nullptr, nullptr}
#define DG_LIN_ENTRY(NAME, BF16, BM, BN, BK, WM, WN, S, GM, STEP, ALONE, BLOCK)                 \
    LinearConfig{NAME, STEP, ALONE, BLOCK, BM, BN, BK, 64 * (WM) * (WN), S, GM,                 \
                 {DG_LIN_FNS(BF16, BM, BN, BK, WM, WN, S, N), DG_LIN_FNS(BF16, BM, BN, BK, WM, WN, S, T), \
                  DG_LIN_FNS(BF16, BM, BN, BK, WM, WN, S, W)}},

const LinearConfig *linear_configs(int dtype, int *count);

// The reduce of `splits` slices of partial sums, in slice order, with the
// epilogue: y (rows x N; rows outside the groups are left alone) or dw
// (groups x M x N).
hipError_t launch_linear_reduce(const LinearArgs &args, bool weight_grad, hipStream_t stream);

// Copies a stored matrix into rows of a 16-byte pitch (gemm_aux.hip).
hipError_t launch_stage_rows(const void *src, int64_t ld, int64_t rows, int64_t cols, int esize,
                             void *dst, int64_t ldd, hipStream_t stream);

// dz and dbias.
struct ActGradArgs {
    const void *dy, *pre;
    void *dz;               // or nullptr
    float *dbias;           // or nullptr
    float *ws;              // per row chunk and column: partial sums of dbias
    const int32_t *offsets;
    int64_t lddy, ldp, lddz;
    int rows, N, groups;
    int act, bf16, pre_bf16;
    int vec;                // rows of dy, pre and dz are 16-byte aligned
    int chunk_rows;         // rows of one chunk of the sums; 0: blocks take whole groups
    int chunks;             // chunks that ws has room for: all that there can be
};
hipError_t launch_act_grad(const ActGradArgs &args, hipStream_t stream);

}  // namespace dg
