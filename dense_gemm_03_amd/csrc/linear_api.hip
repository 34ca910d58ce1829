// C ABI of the linear layers (include/gemm_linear.h): argument checks, choice
// of table entry and slices, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm_internal.hpp"
#include "gemm_linear.h"
#include "linear_configs.hpp"

namespace dg {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;   // as gemm.h
constexpr int64_t kMaxGroups = 65535;

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

// The entry and the slices of the summed axis of one product.
struct Plan {
    int cfg = -1;
    int form = 0;
    int splits = 1;
    int64_t tiles_m = 0;   // row tiles: exact, or (grouped) the most there can be
    int64_t tiles_n = 0;
    int64_t ws_bytes = 0;
};

int index_of(int dtype, int bm, int bn, int form)
{
    int count = 0;
    const LinearConfig *tab = linear_configs(dtype, &count);
    for (int i = 0; i < count; ++i)
        if (tab[i].bm == bm && (bn == 0 || tab[i].bn == bn) && tab[i].fn[form][0] != nullptr) return i;
    return -1;
}

// M x N output tiles of a (the groups') product over a summed extent K.
Plan make_plan(const gemm_linear_params &p, bool wgrad)
{
    Plan pl;
    const int64_t cus = device_compute_units();
    pl.form = wgrad ? FORM_WGRAD : p.transw == GEMM_OP_T ? FORM_T : FORM_N;
    const int64_t groups = std::max<int64_t>(1, p.groups);
    const bool grouped = p.groups > 0;
    // extents of one group's product, its rows at the average
    const int64_t M = wgrad ? (p.transw == GEMM_OP_T ? p.N : p.K) : p.rows;
    const int64_t N = wgrad && p.transw == GEMM_OP_T ? p.K : p.N;
    const int64_t K = wgrad ? ceil_div(p.rows, groups) : p.K;
    int count = 0;
    const LinearConfig *tab = linear_configs(p.dtype, &count);
    // expected row tiles: a group's last tile is half full on average
    auto row_tiles = [&](int bm) {
        return wgrad ? groups * ceil_div(M, bm)
                     : grouped ? std::max<int64_t>(1, M / bm + std::min(groups, M) / 2) : ceil_div(M, bm);
    };
    if (t_cfg >= 0) {
        pl.cfg = t_cfg < count && tab[t_cfg].fn[pl.form][0] != nullptr ? t_cfg : -1;
        if (pl.cfg < 0) return pl;
    } else {
        const int64_t per = wgrad ? M : grouped ? ceil_div(M, groups) : M;
        if (!wgrad && per <= 16 && !(grouped && per > 8)) {
            // strips as wide as still give every compute unit a block
            pl.cfg = index_of(p.dtype, 16, 0, pl.form);
            for (int i = pl.cfg + 1; i > 0 && i < count; ++i)
                if (tab[i].bm == 16 && tab[i].fn[pl.form][0] != nullptr &&
                    row_tiles(16) * ceil_div(N, tab[i].bn) >= (pl.form == FORM_T ? 2 * cus : cus))
                    pl.cfg = i;
        } else if (!wgrad && per <= 32)
            pl.cfg = index_of(p.dtype, 32, p.dtype == GEMM_DTYPE_F32 ? 128 : 256, pl.form);
        else if (row_tiles(256) * ceil_div(N, 256) >= cus * 3 / 4 && (wgrad || per >= 192))
            pl.cfg = index_of(p.dtype, 256, 256, pl.form);
        else if (row_tiles(128) * ceil_div(N, 128) >= cus * 3 / 4 && (wgrad || per >= 96))
            pl.cfg = index_of(p.dtype, 128, 128, pl.form);
        else
            pl.cfg = index_of(p.dtype, 64, 64, pl.form);
        if (pl.cfg < 0) return pl;
    }
    const LinearConfig &c = tab[pl.cfg];
    pl.tiles_n = ceil_div(N, c.bn);
    pl.tiles_m = wgrad ? ceil_div(M, c.bm)
                       : grouped ? M / c.bm + std::min(groups, M) : ceil_div(M, c.bm);
    if (c.stages == 0) return pl;
    const int64_t tiles = row_tiles(c.bm) * pl.tiles_n;
    const int64_t ktiles = ceil_div(K, c.bk);
    int64_t s = 1;
    if (t_split > 0)
        s = t_split;
    else if (tiles > 0 && tiles < cus)
        s = std::min(ceil_div(2 * cus, tiles), ktiles / 4);
    s = std::max<int64_t>(1, std::min<int64_t>(s, std::max<int64_t>(ktiles, 1)));
    s = std::min<int64_t>(s, 64);
    if (!wgrad) s = std::max<int64_t>(1, ceil_div(ktiles, ceil_div(std::max<int64_t>(ktiles, 1), s)));
    pl.splits = (int)s;
    if (s > 1) pl.ws_bytes = s * (wgrad ? groups * M : p.rows) * N * 4;
    return pl;
}

bool aligned16(const void *p, int64_t ld, int64_t stride, int dtype)
{
    const int64_t vec = 16 / size_of(dtype);
    return (uintptr_t)p % 16 == 0 && ld % vec == 0 && stride % vec == 0;
}

int launch_plan(const Plan &pl, int dtype, LinearArgs &a, bool wgrad, void *workspace, hipStream_t stream)
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
    // Blocks per XCD, for all eight: the tiles (or, grouped, the most there can
    // be), rounded up for either list, and room for the pieces of a last round
    // (xcd_piece): at most 3/2 of the slots more.
    const int64_t tiles = pl.tiles_m * pl.tiles_n;
    a.slots = c.bm == 256 && c.bn == 256 && dtype == GEMM_DTYPE_BF16 ? device_compute_units() / 8 : 0;
    const int64_t per = (wgrad ? ceil_div(tiles, 8) * a.groups * pl.splits : tiles * pl.splits / 8 + 2) +
                        ceil_div(a.slots * 3, 2);
    if (per > INT32_MAX / 8) return GEMM_ERR_INVALID_ARG;
    const int64_t blocks = per * 8;
    if (c.fn[pl.form][x16 && w16 ? 0 : 1](a, (int)blocks, stream) != hipSuccess) return GEMM_ERR_HIP;
    if (pl.splits > 1 && launch_linear_reduce(a, wgrad, stream) != hipSuccess) return GEMM_ERR_HIP;
    return GEMM_OK;
}

bool valid_workspace(const void *ws, int64_t bytes, int64_t need)
{
    return need == 0 || (ws != nullptr && (uintptr_t)ws % 16 == 0 && bytes >= need);
}

// Scratch of the bias gradient: one row of N sums per chunk of rows, when
// there is more than one chunk.
int64_t act_grad_chunks(const gemm_linear_params &p)
{
    return p.groups > 0 ? p.rows / kActGradRows + std::min(p.groups, p.rows)
                        : ceil_div(p.rows, kActGradRows);
}

int64_t act_grad_bytes(const gemm_linear_params &p)
{
    if (p.groups == 0 && p.rows <= kActGradRows && p.rows > 0) return 0;
    return std::max<int64_t>(16, act_grad_chunks(p) * p.N * 4);
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
           int64_t workspace_bytes, hipStream_t stream)
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
    gemm_linear_params q = *p;
    if (!sums) q.K = 0;
    const Plan pl = make_plan(q, false);
    if (pl.cfg < 0) return t_cfg >= 0 ? GEMM_ERR_INVALID_ARG : GEMM_ERR_INTERNAL;
    if (!valid_workspace(workspace, workspace_bytes, empty ? 0 : pl.ws_bytes)) return GEMM_ERR_INVALID_ARG;
    if (empty) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    LinearArgs a{};
    a.x = x;
    a.w = w;
    a.offsets = p->groups > 0 ? offsets : nullptr;
    a.ldx = p->ldx;
    a.ldw = p->ldw;
    a.stride_w = p->groups > 0 ? p->stride_w : 0;
    a.stride_bias = p->groups > 0 ? p->stride_bias : 0;
    a.rows = a.M = (int)p->rows;
    a.N = (int)p->N;
    a.K = (int)q.K;
    a.groups = (int)std::max<int64_t>(1, p->groups);
    a.e = EpilogueArgs{y, pre, residual, bias, p->ldy, p->ldr, p->ldp, p->alpha, 1.0f, p->act,
                       p->dtype_y == GEMM_DTYPE_BF16, p->dtype_bias == GEMM_DTYPE_BF16, 0};
    a.e.vec = aligned16(y, p->ldy, 0, p->dtype_y) && (!residual || aligned16(residual, p->ldr, 0, p->dtype_y)) &&
              (!pre || aligned16(pre, p->ldp, 0, p->dtype_y));
    return launch_plan(pl, p->dtype, a, false, workspace, stream);
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
    const int64_t need = dbias && p->N > 0 ? act_grad_bytes(*p) : 0;
    if (!valid_workspace(workspace, workspace_bytes, need)) return GEMM_ERR_INVALID_ARG;
    if (p->N == 0 || (!dz && !dbias) || (p->rows == 0 && !dbias)) return GEMM_OK;
    if (p->groups > 0 && !offsets) return GEMM_ERR_INVALID_ARG;
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
    const int64_t chunks = act_grad_chunks(*p);
    a.chunks = (int)chunks;
    if (chunks * ceil_div(p->N, a.bf16 ? 512 : 256) > INT32_MAX ||
        a.groups * ceil_div(p->N, 256) > INT32_MAX)
        return GEMM_ERR_INVALID_ARG;
    return launch_act_grad(a, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

int weight_grad(const gemm_linear_params *p, const void *x, const void *dz, int64_t lddz,
                const int32_t *offsets, int dtype_dw, float beta, void *dw, void *workspace,
                int64_t workspace_bytes, hipStream_t stream)
{
    if (!valid_sizes(p) || !valid_operands(p) || !known(dtype_dw)) return GEMM_ERR_INVALID_ARG;
    const bool sums = p->rows > 0 && p->alpha != 0.0f, empty = p->K == 0 || p->N == 0;
    if (lddz < std::max<int64_t>(p->N, 1)) return GEMM_ERR_INVALID_ARG;
    if (!empty && (!dw || (sums && (!x || !dz)) || (p->groups > 0 && !offsets))) return GEMM_ERR_INVALID_ARG;
    if (misaligned(x, p->dtype) || misaligned(dz, p->dtype) || misaligned(dw, dtype_dw) ||
        (uintptr_t)offsets % 4)
        return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (!sums) q.rows = 0;
    const Plan pl = make_plan(q, true);
    if (pl.cfg < 0) return t_cfg >= 0 ? GEMM_ERR_INVALID_ARG : GEMM_ERR_INTERNAL;
    if (!valid_workspace(workspace, workspace_bytes, empty ? 0 : pl.ws_bytes)) return GEMM_ERR_INVALID_ARG;
    if (empty) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    const bool t = p->transw == GEMM_OP_T;   // dw^T = dz^T . x
    LinearArgs a{};
    a.x = t ? dz : x;
    a.w = t ? x : dz;
    a.ldx = t ? lddz : p->ldx;
    a.ldw = t ? p->ldx : lddz;
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

}  // namespace
}  // namespace dg

extern "C" {

int64_t gemm_linear_workspace_size(const gemm_linear_params *p)
{
    if (!dg::valid_sizes(p)) return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (p->alpha == 0.0f) q.K = 0;
    return p->rows == 0 || p->N == 0 ? 0 : dg::make_plan(q, false).ws_bytes;
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
    if (!dg::valid_sizes(p)) return GEMM_ERR_INVALID_ARG;
    gemm_linear_params q = *p;
    if (p->alpha == 0.0f) q.rows = 0;
    return p->K == 0 || p->N == 0 ? 0 : dg::make_plan(q, true).ws_bytes;
}

int gemm_linear_weight_grad(const gemm_linear_params *p, const void *x, const void *dz, int64_t lddz,
                            const int32_t *offsets, int dtype_dw, float beta, void *dw,
                            void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return dg::weight_grad(p, x, dz, lddz, offsets, dtype_dw, beta, dw, workspace, workspace_bytes, stream);
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
    return cfg >= 0 ? cfg : dg::t_cfg >= 0 ? GEMM_ERR_INVALID_ARG : GEMM_ERR_INTERNAL;
}

int gemm_linear_force_config(int cfg, int split_k)
{
    dg::t_cfg = cfg < 0 ? -1 : cfg;
    dg::t_split = split_k <= 0 ? 0 : split_k;
    return GEMM_OK;
}

}  // extern "C"
