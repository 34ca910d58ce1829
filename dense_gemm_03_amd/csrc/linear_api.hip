// C ABI of the linear layers (include/gemm_linear.h): argument checks, choice
// of table entry and slices, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "gemm_internal.hpp"
#include "gemm_linear.h"
#include "linear_configs.hpp"
#include "serving.hpp"

namespace dg {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;   // as gemm.h
constexpr int64_t kMaxGroups = 65535;
constexpr int64_t kMaxThreads = UINT32_MAX;      // of one launch

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int size_of(int dtype) { return dtype == GEMM_DTYPE_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == GEMM_DTYPE_F32 || dtype == GEMM_DTYPE_BF16; }
bool misaligned(const void *p, int dtype) { return (uintptr_t)p % (uintptr_t)size_of(dtype) != 0; }

thread_local int t_cfg = -1, t_split = 0;   // gemm_linear_force_config

// Sizes, types and enumerations: what every call checks.
bool valid_sizes(const gemm_linear_params *p)
{
    return p != nullptr && known(p->dtype) && known(p->dtype_y) && known(p->dtype_bias) &&
           (p->transw == GEMM_OP_N || p->transw == GEMM_OP_T) && p->act >= GEMM_ACT_NONE &&
           p->act <= GEMM_ACT_SILU && p->rows >= 0 && p->rows <= kMaxSize && p->N >= 0 &&
           p->N <= kMaxSize && p->K >= 0 && p->K <= kMaxSize && p->groups >= 0 &&
           p->groups <= kMaxGroups;
}

// Leading dimensions and strides of x and w.
bool valid_operands(const gemm_linear_params *p)
{
    const int64_t wrow = p->transw == GEMM_OP_T ? p->K : p->N;
    const int64_t wrows = p->transw == GEMM_OP_T ? p->N : p->K;
    if (p->ldx < std::max<int64_t>(p->K, 1) || p->ldw < std::max<int64_t>(wrow, 1)) return false;
    if (p->ldx > (int64_t(1) << 40) || p->ldw > (int64_t(1) << 40)) return false;
    // the groups' weights do not overlap
    return p->groups <= 1 || wrow == 0 || wrows == 0 ||
           p->stride_w >= (wrows - 1) * p->ldw + wrow;
}

// The entry and the slices of the summed axis of one product, and what it
// needs of the workspace.
struct Plan {
    int cfg = -1;
    int form = 0;
    int splits = 1;
    int64_t tiles_m = 0;   // row tiles: exact, or (grouped) the most there can be
    int64_t tiles_n = 0;
    // copies of x and w (of the second form: x and dz) with 16-byte rows: pitch
    // in elements (0: none) and place in the workspace
    int64_t copy_x = 0, copy_w = 0, at_x = 0, at_w = 0;
    int64_t ws_bytes = 0;
};

// Estimated time in us of entry c on a product of `tiles` output tiles over K,
// cut into s slices: rounds of blocks over the compute units, k-tiles at the
// rate of a full unit or of a block alone, whichever is longer, and the reduce.
// The entries' constants, the reduce's 3.5 us + bytes / 4.6 TB/s and the model's
// form were fitted to timings of every entry in 1 to 16 slices (dense, M 40 to
// 4096, N 256 to 8192, K 512 to 8192, all forms); the pieces' factors and the
// grouped rates come from single shapes.  Against the fastest of all entries and
// slices the choice is, in the mean, 3.1% slower over 417 dense bf16 shapes and
// 1.2% over 363 fp32 ones, 5.2% and 2.6% for grouped y (96 and 84 shapes), but 25%
// and 35% for grouped dw (48 and 42): the bytes of the outputs are not in the
// model, and dw of groups of few rows is mostly those.  With groups the smaller
// bf16 tiles are taken to run a quarter slower: the weights come from HBM and each
// is read by a few row tiles only (12000 rows of 10 groups, 2048 x 2048: 0.58 us per
// k-tile of 128 x 128, against 0.45).
double estimate(const LinearConfig &c, double tiles, bool grouped, bool exact, int64_t out, int64_t K, int64_t s,
                int64_t cus, int es)
{
    const double blocks = tiles * (double)s;
    const int64_t per_cu = std::min<int64_t>(8, int64_t(160 * 1024) / ((int64_t)c.stages * (c.bm + c.bn) * c.bk * es));
    const double ktiles = (double)ceil_div(K, c.bk * s);
    const double step = grouped && es == 2 && c.bm < 256 ? 1.25 * c.step : c.step;
    double busy = std::max(1.0, std::ceil(blocks / (double)cus));   // blocks of the fullest unit
    double rounds = std::ceil(busy / (double)per_cu);
    if (!exact) {                   // a count of tiles that is not known: no steps
        busy = std::max(1.0, blocks / (double)cus + (es == 2 && c.bm == 256 ? 0.2 : 0.3));
        rounds = std::max(1.0, busy / (double)per_cu);
    } else if (es == 2 && c.bm == 256) {   // pieces in the last round (xcd_piece)
        const double whole = std::floor(blocks / (double)cus), rest = blocks - whole * (double)cus;
        busy = whole + (rest <= 0 ? 0.0 : 4 * rest <= cus ? 0.4 : 2 * rest <= cus ? 0.6 : std::max(0.72, rest / (double)cus));
        rounds = whole + (rest > 0 ? 1.0 : 0.0);
    }
    double t = 3.0 + c.block * rounds + ktiles * std::max(step * busy, c.alone * rounds);
    if (s > 1) t += 3.5 + 0.1 * (double)s + (double)s * (double)out * 8.0 / 4.6e6;
    return t;
}

// The same for the kernel for few rows: a compute unit streams 38 KB per us of
// weights and x (measured: 33 to 49), whatever the strip's width.
double estimate_rows(const LinearConfig &c, double tiles, int64_t N, int64_t K, double rows, int64_t cus, int es)
{
    const double busy = std::ceil(std::max(1.0, tiles * (double)ceil_div(N, c.bn)) / (double)cus);
    return 3.3 + busy * ((double)c.bn + std::min(rows, 16.0)) * (double)K * es / 38e3;
}

// Compute units per XCD that pieces of a last round go to (xcd_piece); 0 for
// entries without pieces.
int64_t piece_slots(const LinearConfig &c, int dtype, int64_t cus)
{
    return c.bm == 256 && c.bn == 256 && dtype == GEMM_DTYPE_BF16 ? cus / 8 : 0;
}

// Blocks of an entry's grid.  Per XCD: the tiles (or, grouped, the most there
// can be), rounded up for either list, and room for the pieces of a last round:
// at most 3/4 of the slots more, and one more per group's last row of tiles.
int64_t grid_blocks(int64_t tiles_m, int64_t tiles_n, bool wgrad, int64_t groups, int64_t rows, int64_t splits,
                    int64_t slots)
{
    const int64_t tiles = tiles_m * tiles_n;
    if (tiles > kMaxThreads) return INT64_MAX;   // and the products below stay in 64 bits
    const int64_t lasts = wgrad ? 0 : std::min(groups, rows) * tiles_n * splits;
    return 8 * ((wgrad ? ceil_div(tiles, 8) * groups * splits : tiles * splits / 8 + 2) +
                (slots > 0 ? ceil_div(slots * 3, 4) + lasts / 8 + 2 : 0));
}

Plan find_plan(const gemm_linear_params &p, bool wgrad, int64_t cus)
{
    Plan pl;
    pl.form = wgrad ? FORM_WGRAD : p.transw == GEMM_OP_T ? FORM_T : FORM_N;
    const int64_t groups = std::max<int64_t>(1, p.groups);
    const bool grouped = p.groups > 0, turned = wgrad && p.transw == GEMM_OP_T;
    // extents of one group's product, its rows at the average
    const int64_t M = wgrad ? (turned ? p.N : p.K) : p.rows;
    const int64_t N = turned ? p.K : p.N;
    const int64_t K = wgrad ? ceil_div(p.rows, groups) : p.K;
    const int es = size_of(p.dtype);
    const double per = (double)p.rows / (double)groups;
    // Row tiles to expect.  Of a group's rows the last tile is half full on
    // average; groups of few rows (counts spread like Poisson's) have one
    // unless they are empty.
    auto row_tiles = [&](int64_t bm) -> double {
        if (wgrad) return (double)(groups * ceil_div(M, bm));
        if (!grouped) return (double)ceil_div(M, bm);
        return std::max(std::max(1.0, (double)groups * (1.0 - std::exp(-per))),
                        (double)M / (double)bm + 0.5 * (double)std::min(groups, M));
    };
    const int64_t out = (wgrad ? groups * M : p.rows) * N;   // outputs
    // bf16 operands without 16-byte rows lose the wide direct loads of the
    // tiles: in place, rows at 4-byte boundaries take 1.45 times as long, others
    // 3.5 times (2048^3: 23 us against 32 and 81 to 108).  Where that costs more
    // than copying them into rows of 16-byte pitch first (a launch, and a pass at
    // 3 TB/s over each), they are copied.  fp32 operands lose 10% at most, and
    // the kernel for few rows nothing.
    const int64_t w_ld = wgrad ? p.ldy : p.ldw;
    const int64_t w_rows = wgrad ? p.rows : groups * (p.transw == GEMM_OP_T ? p.N : p.K);
    const int64_t w_cols = wgrad ? p.N : p.transw == GEMM_OP_T ? p.K : p.N;
    const int64_t px = ceil_div(p.K, 8) * 8, pw = ceil_div(w_cols, 8) * 8;
    const bool bf16 = p.dtype == GEMM_DTYPE_BF16 && K > 0 && out > 0;
    const bool x_odd = bf16 && p.ldx % 8 != 0;
    const bool w_odd = bf16 && (w_ld % 8 != 0 || (!wgrad && groups > 1 && p.stride_w % 8 != 0));
    const double in_place = !(x_odd || w_odd) ? 1.0 : ((p.ldx | w_ld) & 1) != 0 ? 3.5 : 1.45;
    // the groups' weights have to be one matrix for that; a forced entry runs in place
    const bool may_copy = (x_odd || w_odd) && t_cfg < 0 &&
                          (!w_odd || wgrad || groups == 1 || p.stride_w == w_rows / groups * p.ldw);
    const double copying = (x_odd ? 3.0 + (double)p.rows * (double)px * 4.0 / 3e6 : 0.0) +
                           (w_odd ? 3.0 + (double)w_rows * (double)pw * 4.0 / 3e6 : 0.0);

    // An entry's time t, or that of the weights (for dw, of x and dz) from HBM at
    // 4.7 TB/s, whichever is longer, and a part of the other: a tenth, or half
    // where two stages are all that covers HBM's latency (512 x 8192 x 8192, one
    // 128 x 128 block per unit: 106 us, 76 by the cached rate; 256 x 256: 81).
    const double stream = (wgrad ? (double)p.rows * (double)(p.K + p.N)
                                 : row_tiles((int64_t(1) << 31)) * (double)K * (double)N) * es / 4.7e6;
    auto with_stream = [&](double t, double part) { return std::max(stream, t) + part * std::min(stream, t); };

    auto tiles_m = [&](const LinearConfig &c) {
        return !wgrad && grouped ? M / c.bm + std::min(groups, M) : ceil_div(M, c.bm);
    };
    auto launchable = [&](const LinearConfig &c, int64_t s) {
        return grid_blocks(tiles_m(c), ceil_div(N, c.bn), wgrad, groups, p.rows, s, piece_slots(c, p.dtype, cus)) <=
               kMaxThreads / c.threads;
    };

    int count = 0;
    const LinearConfig *tab = linear_configs(p.dtype, &count);
    double best = 0.0;
    bool copies = false;
    for (int i = 0; i < count; ++i) {
        const LinearConfig &c = tab[i];
        if (c.fn[pl.form][0] == nullptr || (t_cfg >= 0 && i != t_cfg)) continue;
        if (c.stages == 0) {
            const double t = with_stream(estimate_rows(c, row_tiles(16), N, K, per, cus, es), 0.1);
            if (launchable(c, 1) && (pl.cfg < 0 || t < best)) {
                pl.cfg = i;
                pl.splits = 1;
                best = t;
                copies = false;
            }
            continue;
        }
        const int64_t ktiles = std::max<int64_t>(1, ceil_div(K, c.bk));
        static const int slices[] = {1, 2, 3, 4, 6, 8, 12, 16};
        for (int want : slices) {
            if (t_split > 0) want = t_split;
            int64_t s = std::min<int64_t>(want, std::min<int64_t>(ktiles, 64));
            if (!wgrad) s = ceil_div(ktiles, ceil_div(ktiles, s));   // every slice has a k-tile
            const double whole = with_stream(estimate(c, row_tiles(c.bm) * (double)ceil_div(N, c.bn), grouped,
                                                      wgrad || !grouped, out, K, s, cus, es),
                                             es == 2 && c.stages == 2 && c.bm < 256 ? 0.5 : 0.1);
            const bool copied = may_copy && whole + copying < whole * in_place;
            const double t = copied ? whole + copying : whole * in_place;
            if (launchable(c, s) && (pl.cfg < 0 || t < best)) {
                pl.cfg = i;
                pl.splits = (int)s;
                best = t;
                copies = copied;
            }
            if (t_split > 0 || want >= ktiles) break;
        }
    }
    if (pl.cfg < 0) return pl;
    const LinearConfig &c = tab[pl.cfg];
    pl.tiles_n = ceil_div(N, c.bn);
    pl.tiles_m = tiles_m(c);
    if (pl.splits > 1) pl.ws_bytes = (pl.splits * out * 4 + 255) / 256 * 256;

    if (copies && x_odd) {
        pl.copy_x = px;
        pl.at_x = pl.ws_bytes;
        pl.ws_bytes += (p.rows * px * 2 + 255) / 256 * 256;
    }
    if (copies && w_odd) {
        pl.copy_w = pw;
        pl.at_w = pl.ws_bytes;
        pl.ws_bytes += w_rows * pw * 2;
    }
    return pl;
}

// Plans by their parameters, a few per thread: a call asks for the workspace
// size first, and the next call is often the same.
Plan make_plan(const gemm_linear_params &p, bool wgrad)
{
    struct Known {
        bool set = false, wgrad = false;
        int cfg = 0, split = 0;
        int64_t cus = 0;
        gemm_linear_params p{};
        Plan plan;
    };
    thread_local Known known[16];
    thread_local unsigned next = 0;
    const int64_t cus = device_compute_units();
    for (Known &k : known)
        if (k.set && k.wgrad == wgrad && k.cfg == t_cfg && k.split == t_split && k.cus == cus &&
            std::memcmp(&k.p, &p, sizeof p) == 0)
            return k.plan;
    Known &k = known[next++ % 16];
    k = Known{true, wgrad, t_cfg, t_split, cus, p, find_plan(p, wgrad, cus)};
    return k.plan;
}

bool aligned16(const void *p, int64_t ld, int64_t stride, int dtype)
{
    const int64_t vec = 16 / size_of(dtype);
    return (uintptr_t)p % 16 == 0 && ld % vec == 0 && stride % vec == 0;
}

// Copies `rows` rows of `cols` bf16 values to rows of `pitch` in the workspace.
int copy_rows(const void **m, int64_t *ld, int64_t rows, int64_t cols, int64_t pitch, void *workspace,
              int64_t at, hipStream_t stream)
{
    void *to = static_cast<char *>(workspace) + at;
    if (launch_stage_rows(*m, *ld, rows, cols, 2, to, pitch, stream) != hipSuccess) return GEMM_ERR_HIP;
    *m = to;
    *ld = pitch;
    return GEMM_OK;
}

// With `ad` (first two forms): an adapter per row.
int launch_plan(const Plan &pl, int dtype, LinearArgs &a, bool wgrad, void *workspace, hipStream_t stream,
                const AdapterArgs *ad = nullptr)
{
    int count = 0;
    const LinearConfig &c = linear_configs(dtype, &count)[pl.cfg];
    const bool x16 = aligned16(a.x, a.ldx, 0, dtype);
    const bool w16 = aligned16(a.w, a.ldw, a.stride_w, dtype);
    const int vec = 16 / size_of(dtype);
    // outer-contiguous rows are read in whole 16-byte chunks past the edge:
    // inside the row's pitch, or on the page of the row's last element
    a.m_load = wgrad && x16 ? (int)(ceil_div(a.M, vec) * vec) : a.M;
    a.n_load = pl.form != FORM_T && w16 ? (int)(ceil_div(a.N, vec) * vec) : a.N;
    const int64_t es = size_of(dtype);
    const int64_t x_rows = wgrad ? c.bk : c.bm, w_rows = pl.form == FORM_T ? c.bn : c.bk;
    a.direct_ok = x_rows * a.ldx * es < (int64_t(1) << 32) && w_rows * a.ldw * es < (int64_t(1) << 32);
    a.tiles_n = (int)pl.tiles_n;
    a.tiles_m = (int)pl.tiles_m;
    a.splits = pl.splits;
    a.group_m = c.group_m;
    a.k_per_split = (int)(ceil_div(ceil_div(a.K, c.bk), pl.splits) * c.bk);
    a.ws = pl.splits > 1 ? static_cast<float *>(workspace) : nullptr;
    a.slots = (int)piece_slots(c, dtype, device_compute_units());
    const int64_t blocks = grid_blocks(pl.tiles_m, pl.tiles_n, wgrad, a.groups, a.rows, pl.splits, a.slots);
    const int odd = x16 && w16 ? 0 : 1;
    const hipError_t err = ad != nullptr ? c.adapted[pl.form][odd](AdaptedArgs{a, *ad}, (int)blocks, stream)
                                         : c.fn[pl.form][odd](a, (int)blocks, stream);
    if (err != hipSuccess) return GEMM_ERR_HIP;
    if (pl.splits > 1 && launch_linear_reduce(a, wgrad, stream) != hipSuccess) return GEMM_ERR_HIP;
    return GEMM_OK;
}

bool valid_workspace(const void *ws, int64_t bytes, int64_t need)
{
    return need == 0 || (ws != nullptr && (uintptr_t)ws % 16 == 0 && bytes >= need);
}

// Scratch of the bias gradient.  Up to 128 rows per group on average and 1024 in
// all, a block walks all of a group's rows and its sums are the result, without
// a second launch (28 groups of 26 rows, whole backward pass: 15.0 us against
// 21.6; but 484 rows of one: 31 against 26.5).  Beyond, chunks of rows, a row of
// N sums each: 64 rows; 32 with groups, whose last chunks are short (16 groups,
// 8192 x 4096: 58 us against 64; one group: 50 against 44); 16 where 64 would
// leave fewer than two blocks per compute unit (777 x 1025 fp32: 19 us with 65
// blocks of 64 rows).
int act_grad_rows(const gemm_linear_params &p)
{
    const int64_t blocks = ceil_div(p.rows, 64) * ceil_div(p.N, p.dtype == GEMM_DTYPE_F32 ? 256 : 512);
    if (p.rows <= 1024 && p.rows <= 128 * std::max<int64_t>(1, p.groups)) return 0;
    return blocks < 512 ? 16 : p.groups > 0 ? 32 : 64;
}

int64_t act_grad_chunks(const gemm_linear_params &p)
{
    const int64_t rows = act_grad_rows(p);
    if (rows == 0) return 0;
    return p.groups > 0 ? p.rows / rows + std::min(p.groups, p.rows) : ceil_div(p.rows, rows);
}

int64_t act_grad_bytes(const gemm_linear_params &p) { return act_grad_chunks(p) * p.N * 4; }

// Whether launch_act_grad's grids hold in a launch: blocks of 16 bytes per lane
// (below 1024 of those there may be 8 times as many, still few), and the reduce.
bool act_grad_fits(const gemm_linear_params &p, bool dbias)
{
    const bool whole = act_grad_rows(p) == 0;
    const int64_t groups = std::max<int64_t>(1, p.groups);
    const int64_t blocks = (whole ? groups : act_grad_chunks(p)) * ceil_div(p.N, p.dtype == GEMM_DTYPE_F32 ? 256 : 512);
    return blocks <= kMaxThreads / (whole ? 1024 : 256) &&
           (!dbias || whole || groups * ceil_div(p.N, 64) <= kMaxThreads / 256);
}

int need_device()
{
    int device = -1;
    if (hipGetDevice(&device) == hipSuccess) return GEMM_OK;
    (void)hipGetLastError();
    return GEMM_ERR_NO_DEVICE;
}

int linear(const gemm_linear_params *p, const void *x, const void *w, const int32_t *offsets,
           const void *bias, const void *residual, void *pre, void *y, void *workspace,
           int64_t workspace_bytes, hipStream_t stream, const AdapterArgs *ad = nullptr,
           const AdapterDownArgs *down = nullptr)
{
    if (!valid_sizes(p) || !valid_operands(p)) return GEMM_ERR_INVALID_ARG;
    const int64_t nrow = std::max<int64_t>(p->N, 1);
    const bool sums = p->K > 0 && p->alpha != 0.0f;   // else x and w are not read
    const bool empty = p->rows == 0 || p->N == 0;
    if (p->ldy < nrow || (residual && p->ldr < nrow) || (pre && p->ldp < nrow)) return GEMM_ERR_INVALID_ARG;
    if (!empty && (!y || (sums && (!x || !w)) || (p->groups > 0 && !offsets))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(x, p->dtype) || misaligned(w, p->dtype) || misaligned(bias, p->dtype_bias) ||
        misaligned(residual, p->dtype_y) || misaligned(pre, p->dtype_y) || misaligned(y, p->dtype_y) ||
        (uintptr_t)offsets % 4)
        return GEMM_ERR_INVALID_ARG;
    if (p->groups > 1 && bias && p->stride_bias < p->N) return GEMM_ERR_INVALID_ARG;
    // in place: row r of y lies over row r of the residual and no other
    if (residual && residual == y && p->rows > 1 && p->ldr != p->ldy) return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (!sums) q.K = 0;
    const Plan pl = make_plan(q, false);
    if (pl.cfg < 0) return GEMM_ERR_INVALID_ARG;   // no entry, or no forced one, for this form and size
    if (!valid_workspace(workspace, workspace_bytes, empty ? 0 : pl.ws_bytes)) return GEMM_ERR_INVALID_ARG;
    if (empty) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    if (down && launch_adapter_down(*down, p->dtype == GEMM_DTYPE_BF16, stream) != hipSuccess) return GEMM_ERR_HIP;
    LinearArgs a{};
    a.x = x;
    a.w = w;
    a.ldx = p->ldx;
    a.ldw = p->ldw;
    a.stride_w = p->groups > 0 ? p->stride_w : 0;
    if (pl.copy_x) {
        const int rc = copy_rows(&a.x, &a.ldx, p->rows, p->K, pl.copy_x, workspace, pl.at_x, stream);
        if (rc != GEMM_OK) return rc;
    }
    if (pl.copy_w) {
        const int64_t rows = p->transw == GEMM_OP_T ? p->N : p->K;
        const int rc = copy_rows(&a.w, &a.ldw, rows * std::max<int64_t>(1, p->groups),
                                 p->transw == GEMM_OP_T ? p->K : p->N, pl.copy_w, workspace, pl.at_w, stream);
        if (rc != GEMM_OK) return rc;
        if (p->groups > 0) a.stride_w = rows * pl.copy_w;
    }
    a.offsets = p->groups > 0 ? offsets : nullptr;
    a.stride_bias = p->groups > 0 ? p->stride_bias : 0;
    a.rows = a.M = (int)p->rows;
    a.N = (int)p->N;
    a.K = (int)q.K;
    a.groups = (int)std::max<int64_t>(1, p->groups);
    a.e = EpilogueArgs{y, pre, residual, bias, p->ldy, p->ldr, p->ldp, p->alpha, 1.0f, p->act,
                       p->dtype_y == GEMM_DTYPE_BF16, p->dtype_bias == GEMM_DTYPE_BF16, 0};
    a.e.vec = aligned16(y, p->ldy, 0, p->dtype_y) && (!residual || aligned16(residual, p->ldr, 0, p->dtype_y)) &&
              (!pre || aligned16(pre, p->ldp, 0, p->dtype_y));
    return launch_plan(pl, p->dtype, a, false, workspace, stream, ad);
}

int act_grad(const gemm_linear_params *p, const void *dy, int64_t lddy, const void *pre,
             const int32_t *offsets, void *dz, int64_t lddz, float *dbias, void *workspace,
             int64_t workspace_bytes, hipStream_t stream)
{
    if (!valid_sizes(p)) return GEMM_ERR_INVALID_ARG;
    const int64_t nrow = std::max<int64_t>(p->N, 1);
    const bool act = p->act != GEMM_ACT_NONE, empty = p->rows == 0 || p->N == 0;
    if (lddy < nrow || (dz && lddz < nrow) || (act && p->ldp < nrow)) return GEMM_ERR_INVALID_ARG;
    if (!empty && (!dy || (act && !pre) || (p->groups > 0 && !offsets))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(dy, p->dtype) || misaligned(dz, p->dtype) || misaligned(pre, p->dtype_y) ||
        (uintptr_t)dbias % 4 || (uintptr_t)offsets % 4)
        return GEMM_ERR_INVALID_ARG;
    if (dz && dz == dy && p->rows > 1 && lddz != lddy) return GEMM_ERR_INVALID_ARG;   // as residual and y
    const int64_t need = dbias && p->N > 0 ? act_grad_bytes(*p) : 0;
    if (!valid_workspace(workspace, workspace_bytes, need)) return GEMM_ERR_INVALID_ARG;
    if (p->N == 0 || (!dz && !dbias) || (p->rows == 0 && !dbias)) return GEMM_OK;
    if ((p->groups > 0 && !offsets) || !act_grad_fits(*p, dbias != nullptr)) return GEMM_ERR_INVALID_ARG;
    if (const int rc = need_device()) return rc;
    ActGradArgs a{};
    a.dy = dy;
    a.pre = act ? pre : nullptr;
    a.dz = dz;
    a.dbias = dbias;
    a.ws = need > 0 ? static_cast<float *>(workspace) : nullptr;
    a.offsets = p->groups > 0 ? offsets : nullptr;
    a.lddy = lddy;
    a.ldp = p->ldp;
    a.lddz = lddz;
    a.rows = (int)p->rows;
    a.N = (int)p->N;
    a.groups = (int)std::max<int64_t>(1, p->groups);
    a.act = p->act;
    a.bf16 = p->dtype == GEMM_DTYPE_BF16;
    a.pre_bf16 = p->dtype_y == GEMM_DTYPE_BF16;
    a.vec = aligned16(dy, lddy, 0, p->dtype) && (!dz || aligned16(dz, lddz, 0, p->dtype)) &&
            (!act || p->dtype_y != p->dtype || aligned16(pre, p->ldp, 0, p->dtype_y));
    a.chunks = (int)act_grad_chunks(*p);
    a.chunk_rows = act_grad_rows(*p);
    return launch_act_grad(a, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

int weight_grad(const gemm_linear_params *p, const void *x, const void *dz, const int32_t *offsets,
                int dtype_dw, float beta, void *dw, void *workspace, int64_t workspace_bytes,
                hipStream_t stream)
{
    if (!valid_sizes(p) || !valid_operands(p) || !known(dtype_dw)) return GEMM_ERR_INVALID_ARG;
    const bool sums = p->rows > 0 && p->alpha != 0.0f, empty = p->K == 0 || p->N == 0;
    if (p->ldy < std::max<int64_t>(p->N, 1)) return GEMM_ERR_INVALID_ARG;
    if (!empty && (!dw || (sums && (!x || !dz)) || (p->groups > 0 && !offsets))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(x, p->dtype) || misaligned(dz, p->dtype) || misaligned(dw, dtype_dw) ||
        (uintptr_t)offsets % 4)
        return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (!sums) q.rows = 0;
    const Plan pl = make_plan(q, true);
    if (pl.cfg < 0) return GEMM_ERR_INVALID_ARG;   // no entry, or no forced one, for this form and size
    if (!valid_workspace(workspace, workspace_bytes, empty ? 0 : pl.ws_bytes)) return GEMM_ERR_INVALID_ARG;
    if (empty) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    const bool t = p->transw == GEMM_OP_T;   // dw^T = dz^T . x
    int64_t ldx = p->ldx, lddz = p->ldy;
    if (pl.copy_x) {
        const int rc = copy_rows(&x, &ldx, p->rows, p->K, pl.copy_x, workspace, pl.at_x, stream);
        if (rc != GEMM_OK) return rc;
    }
    if (pl.copy_w) {
        const int rc = copy_rows(&dz, &lddz, p->rows, p->N, pl.copy_w, workspace, pl.at_w, stream);
        if (rc != GEMM_OK) return rc;
    }
    LinearArgs a{};
    a.x = t ? dz : x;
    a.w = t ? x : dz;
    a.ldx = t ? lddz : ldx;
    a.ldw = t ? ldx : lddz;
    a.offsets = p->groups > 0 ? offsets : nullptr;
    a.stride_c = p->groups > 0 ? p->stride_w : 0;
    a.rows = (int)q.rows;
    a.K = (int)q.rows;
    a.M = (int)(t ? p->N : p->K);
    a.N = (int)(t ? p->K : p->N);
    a.groups = (int)std::max<int64_t>(1, p->groups);
    a.e = EpilogueArgs{dw, nullptr, beta != 0.0f ? dw : nullptr, nullptr, p->ldw, p->ldw, 0, p->alpha,
                       beta, GEMM_ACT_NONE, dtype_dw == GEMM_DTYPE_BF16, 0, 0};
    a.e.vec = aligned16(dw, p->ldw, a.stride_c, dtype_dw);
    return launch_plan(pl, p->dtype, a, true, workspace, stream);
}

// The pieces of the backward pass and their places in the workspace: dz first,
// then scratch that they take in turn (they run one after another).
struct GradParts {
    gemm_linear_params act, dx, dw;
    int64_t lddz = 0, dz_bytes = 0, act_bytes = 0, dx_bytes = 0, dw_bytes = 0, total = 0;
    bool need_act = false, need_dz = false;
    bool forms = true;   // false: no entry, or not the forced one, has a form and its size
};

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

GradParts grad_parts(const gemm_linear_params &p, const gemm_linear_grad_outputs &o, bool dx, bool dw, bool db)
{
    GradParts g;
    const int64_t vec = 16 / size_of(p.dtype);
    g.need_dz = p.act != GEMM_ACT_NONE && (dx || dw);
    g.need_act = g.need_dz || db;
    g.lddz = g.need_dz ? std::max<int64_t>(vec, ceil_div(p.N, vec) * vec) : p.ldy;
    g.dz_bytes = g.need_dz ? round16(p.rows * g.lddz * size_of(p.dtype)) : 0;
    g.act = p;
    g.dx = p;
    g.dx.dtype_y = o.dtype_dx;
    g.dx.dtype_bias = GEMM_DTYPE_F32;
    g.dx.transw = p.transw == GEMM_OP_T ? GEMM_OP_N : GEMM_OP_T;
    g.dx.act = GEMM_ACT_NONE;
    g.dx.N = p.K;
    g.dx.K = p.N;
    g.dx.ldx = g.lddz;
    g.dx.ldy = o.lddx;
    g.dx.ldr = g.dx.ldp = 0;
    g.dx.stride_bias = 0;
    g.dw = p;
    g.dw.act = GEMM_ACT_NONE;
    g.dw.ldy = g.lddz;
    g.dw.ldw = o.lddw;
    g.dw.stride_w = o.stride_dw;
    const bool rows = p.rows > 0;
    g.act_bytes = db && p.N > 0 ? round16(act_grad_bytes(g.act)) : 0;
    gemm_linear_params q = g.dx;
    if (p.alpha == 0.0f) q.K = 0;
    if (dx) {
        const Plan pl = make_plan(q, false);
        g.forms = pl.cfg >= 0;
        g.dx_bytes = rows && p.K > 0 ? round16(pl.ws_bytes) : 0;
    }
    q = g.dw;
    if (p.alpha == 0.0f) q.rows = 0;
    if (dw) {
        const Plan pl = make_plan(q, true);
        g.forms = g.forms && pl.cfg >= 0;
        g.dw_bytes = p.K > 0 && p.N > 0 ? round16(pl.ws_bytes) : 0;
    }
    g.total = g.dz_bytes + std::max(std::max(g.act_bytes, g.dx_bytes), g.dw_bytes);
    return g;
}

// Sizes, types and leading dimensions of a backward pass that forms dx and dw if asked to.
bool valid_backward(const gemm_linear_params *p, const gemm_linear_grad_outputs *o, bool dx, bool dw)
{
    if (!valid_sizes(p) || o == nullptr || !known(o->dtype_dx) || !known(o->dtype_dw) || !valid_operands(p) ||
        p->ldy < std::max<int64_t>(p->N, 1) || (dx && o->lddx < std::max<int64_t>(p->K, 1)))
        return false;
    gemm_linear_params q = *p;   // dw lies as w does
    q.ldw = o->lddw;
    q.stride_w = o->stride_dw;
    return !dw || valid_operands(&q);
}

int grad(const gemm_linear_params *p, const gemm_linear_grad_outputs *o, const void *dy, const void *x,
         const void *w, const int32_t *offsets, const void *pre, void *dx, void *dw, float *dbias,
         void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    if (!valid_backward(p, o, dx != nullptr, dw != nullptr)) return GEMM_ERR_INVALID_ARG;
    const GradParts g = grad_parts(*p, *o, dx != nullptr, dw != nullptr, dbias != nullptr);
    if (!g.forms || !valid_workspace(workspace, workspace_bytes, g.total)) return GEMM_ERR_INVALID_ARG;
    // what the parts check before they launch, checked for all of them before the first
    const bool some = p->rows > 0 && p->N > 0, sums = p->alpha != 0.0f;
    if ((g.need_act && p->act != GEMM_ACT_NONE && (p->ldp < std::max<int64_t>(p->N, 1) || (some && !pre))) ||
        (some && !dy) || (p->groups > 0 && !offsets) || misaligned(dy, p->dtype) || misaligned(pre, p->dtype_y) ||
        (uintptr_t)dbias % 4 || (uintptr_t)offsets % 4 || (g.need_act && !act_grad_fits(*p, dbias != nullptr)))
        return GEMM_ERR_INVALID_ARG;
    if (dx && (misaligned(dx, o->dtype_dx) || misaligned(w, p->dtype) || (some && p->K > 0 && sums && !w)))
        return GEMM_ERR_INVALID_ARG;
    if (dw && (misaligned(dw, o->dtype_dw) || misaligned(x, p->dtype) || (some && p->K > 0 && sums && !x)))
        return GEMM_ERR_INVALID_ARG;
    void *dz = g.need_dz ? workspace : const_cast<void *>(dy);
    void *scratch = workspace ? static_cast<char *>(workspace) + g.dz_bytes : nullptr;
    if (g.need_act) {
        const int rc = act_grad(&g.act, dy, p->ldy, pre, offsets, g.need_dz ? dz : nullptr, g.lddz, dbias,
                                scratch, g.act_bytes, stream);
        if (rc != GEMM_OK) return rc;
    }
    if (dx) {
        const int rc = linear(&g.dx, dz, w, offsets, nullptr, nullptr, nullptr, dx, scratch, g.dx_bytes, stream);
        if (rc != GEMM_OK) return rc;
    }
    if (dw) return weight_grad(&g.dw, x, dz, offsets, o->dtype_dw, o->beta, dw, scratch, g.dw_bytes, stream);
    return GEMM_OK;
}

}  // namespace

bool adapter_sums_allowed(const gemm_linear_params *p)
{
    if (!valid_sizes(p)) return false;
    const Plan pl = make_plan(*p, false);
    int count = 0;
    if (pl.cfg < 0) return false;
    const LinearConfig &c = linear_configs(p->dtype, &count)[pl.cfg];
    return c.bm <= 64 && c.bn <= 64;
}

int linear_with_adapters(const gemm_linear_params *p, const AdapterDownArgs *down, const AdapterArgs *ad,
                         const void *x, const void *w, const void *bias, const void *residual, void *y,
                         void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return linear(p, x, w, nullptr, bias, residual, nullptr, y, workspace, workspace_bytes, stream, ad, down);
}

}  // namespace dg

extern "C" {

int64_t gemm_linear_grad_workspace_size(const gemm_linear_params *p, const gemm_linear_grad_outputs *o, int dx,
                                        int dw, int dbias)
{
    if (!dg::valid_backward(p, o, dx != 0, dw != 0)) return GEMM_ERR_INVALID_ARG;
    const dg::GradParts g = dg::grad_parts(*p, *o, dx != 0, dw != 0, dbias != 0);
    return g.forms ? g.total : GEMM_ERR_INVALID_ARG;
}

int gemm_linear_grad(const gemm_linear_params *p, const gemm_linear_grad_outputs *o, const void *dy,
                     const void *x, const void *w, const int32_t *offsets, const void *pre, void *dx,
                     void *dw, float *dbias, void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return dg::grad(p, o, dy, x, w, offsets, pre, dx, dw, dbias, workspace, workspace_bytes, stream);
}

int64_t gemm_linear_workspace_size(const gemm_linear_params *p)
{
    if (!dg::valid_sizes(p) || !dg::valid_operands(p)) return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (p->alpha == 0.0f) q.K = 0;
    const dg::Plan pl = dg::make_plan(q, false);
    if (pl.cfg < 0) return GEMM_ERR_INVALID_ARG;
    return p->rows == 0 || p->N == 0 ? 0 : pl.ws_bytes;
}

int gemm_linear(const gemm_linear_params *p, const void *x, const void *w, const int32_t *offsets,
                const void *bias, const void *residual, void *pre, void *y, void *workspace,
                int64_t workspace_bytes, hipStream_t stream)
{
    return dg::linear(p, x, w, offsets, bias, residual, pre, y, workspace, workspace_bytes, stream);
}

int64_t gemm_linear_act_grad_workspace_size(const gemm_linear_params *p)
{
    if (!dg::valid_sizes(p)) return GEMM_ERR_INVALID_ARG;
    return p->N == 0 ? 0 : dg::act_grad_bytes(*p);
}

int gemm_linear_act_grad(const gemm_linear_params *p, const void *dy, int64_t lddy, const void *pre,
                         const int32_t *offsets, void *dz, int64_t lddz, float *dbias,
                         void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return dg::act_grad(p, dy, lddy, pre, offsets, dz, lddz, dbias, workspace, workspace_bytes, stream);
}

int64_t gemm_linear_weight_grad_workspace_size(const gemm_linear_params *p)
{
    if (!dg::valid_sizes(p) || !dg::valid_operands(p) || p->ldy < std::max<int64_t>(p->N, 1))
        return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (p->alpha == 0.0f) q.rows = 0;
    const dg::Plan pl = dg::make_plan(q, true);
    if (pl.cfg < 0) return GEMM_ERR_INVALID_ARG;
    return p->K == 0 || p->N == 0 ? 0 : pl.ws_bytes;
}

int gemm_linear_weight_grad(const gemm_linear_params *p, const void *x, const void *dz,
                            const int32_t *offsets, int dtype_dw, float beta, void *dw,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return dg::weight_grad(p, x, dz, offsets, dtype_dw, beta, dw, workspace, workspace_bytes, stream);
}

int gemm_linear_num_configs(int dtype)
{
    if (!dg::known(dtype)) return GEMM_ERR_INVALID_ARG;
    int count = 0;
    (void)dg::linear_configs(dtype, &count);
    return count;
}

const char *gemm_linear_config_name(int dtype, int cfg)
{
    const int count = gemm_linear_num_configs(dtype);
    int n = 0;
    return cfg >= 0 && cfg < count ? dg::linear_configs(dtype, &n)[cfg].name : nullptr;
}

int gemm_linear_config_forms(int dtype, int cfg)
{
    const int count = gemm_linear_num_configs(dtype);
    if (cfg < 0 || cfg >= count) return GEMM_ERR_INVALID_ARG;
    int n = 0, mask = 0;
    for (int f = 0; f < 3; ++f)
        if (dg::linear_configs(dtype, &n)[cfg].fn[f][0] != nullptr) mask |= 1 << f;
    return mask;
}

int gemm_linear_select_config(const gemm_linear_params *p, int weight_grad)
{
    if (!dg::valid_sizes(p)) return GEMM_ERR_INVALID_ARG;
    const int cfg = dg::make_plan(*p, weight_grad != 0).cfg;
    return cfg >= 0 ? cfg : GEMM_ERR_INVALID_ARG;
}

int gemm_linear_force_config(int cfg, int split_k)
{
    dg::t_cfg = cfg < 0 ? -1 : cfg;
    dg::t_split = split_k <= 0 ? 0 : split_k;
    return GEMM_OK;
}

}  // extern "C"
