// C ABI of gemm_serving.h: argument checks, choice of variants, launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gemm_internal.hpp"
#include "gemm_serving.h"
#include "serving.hpp"

namespace dg {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;   // as gemm.h
constexpr int64_t kMaxLd = int64_t(1) << 40;
constexpr float kMaxScale = 0x1p64f;   // its products with log2 e and with a gradient are numbers

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int size_of(int dtype) { return dtype == GEMM_DTYPE_F32 ? 4 : 2; }
bool known(int dtype) { return dtype == GEMM_DTYPE_F32 || dtype == GEMM_DTYPE_BF16; }
bool in_range(int64_t n) { return n >= 0 && n <= kMaxSize; }
bool misaligned(const void *p, int size) { return (uintptr_t)p % (uintptr_t)size != 0; }
bool valid_ld(int64_t ld, int64_t row) { return ld >= std::max<int64_t>(row, 1) && ld <= kMaxLd; }

bool valid_workspace(const void *ws, int64_t bytes, int64_t need)
{
    return need == 0 || (ws != nullptr && (uintptr_t)ws % 16 == 0 && bytes >= need);
}

int need_device()
{
    int device = -1;
    if (hipGetDevice(&device) == hipSuccess) return GEMM_OK;
    (void)hipGetLastError();
    return GEMM_ERR_NO_DEVICE;
}

// ------------------------------------------------------ log probabilities --

bool valid(const gemm_log_probs_params *p)
{
    return p != nullptr && known(p->dtype) && in_range(p->rows) && in_range(p->vocab) && p->vocab >= 1 &&
           p->top >= 0 && p->top <= 64 && p->top <= p->vocab && p->scale > 0.0f && p->scale <= kMaxScale &&
           valid_ld(p->ld, p->vocab);
}

// How a row's chunks are dealt out: waves of a team, parts.
struct Shares {
    int team, parts, part_chunks;
};

Shares shares_of(const gemm_log_probs_params &p)
{
    const int64_t vec = 16 / size_of(p.dtype);
    const int64_t chunks = ceil_div(p.vocab + vec - 1, log_probs_chunk());   // one more where a row starts off a boundary
    // From 8 rows per unit on each row has a wave of its own, fewer are cut so that there
    // are 8 waves per unit (4001 x 50021 bf16, 5 alternatives: 99 us with this bound, 118
    // with one of 16, which cuts those rows, 101 with 4).
    const int64_t waves = 8 * (int64_t)device_compute_units();
    Shares s{1, 1, (int)chunks};
    if (p.rows >= waves || chunks == 1) return s;
    s.team = 4;
    const int64_t parts = std::min(ceil_div(chunks, 4), std::max<int64_t>(1, waves / (4 * std::max<int64_t>(1, p.rows))));
    s.part_chunks = (int)ceil_div(chunks, parts);
    s.parts = (int)ceil_div(chunks, s.part_chunks);
    return s;
}

int64_t log_probs_bytes(const gemm_log_probs_params &p)
{
    const Shares s = shares_of(p);
    return s.parts == 1 ? 0 : p.rows * s.parts * (16 + 8 * (int64_t)p.top);
}

int log_probs(const gemm_log_probs_params *p, const void *logits, const int32_t *tokens, float *logprob,
              float *entropy, float *stats, int32_t *top_ids, float *top_logprobs, void *workspace,
              int64_t workspace_bytes, hipStream_t stream)
{
    if (!valid(p)) return GEMM_ERR_INVALID_ARG;
    const int64_t need = log_probs_bytes(*p);
    if (p->rows > 0 && (!logits || (tokens != nullptr) != (logprob != nullptr) || (p->top > 0 && !top_ids) ||
                        !valid_workspace(workspace, workspace_bytes, need)))
        return GEMM_ERR_INVALID_ARG;
    if (misaligned(logits, size_of(p->dtype)) || misaligned(tokens, 4) || misaligned(logprob, 4) ||
        misaligned(entropy, 4) || misaligned(stats, 4) || misaligned(top_ids, 4) || misaligned(top_logprobs, 4))
        return GEMM_ERR_INVALID_ARG;
    if (p->rows == 0) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    const Shares s = shares_of(*p);
    LogProbsArgs a{};
    a.logits = logits;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.stats = stats;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.ld = p->ld;
    a.rows = p->rows;
    a.vocab = (int)p->vocab;
    a.top = p->top;
    a.scale = p->scale;
    a.parts = s.parts;
    a.part_chunks = s.part_chunks;
    a.team = s.team;
    if (need > 0) {
        a.ws = static_cast<float *>(workspace);
        a.ws_keys = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + p->rows * s.parts * 16);
    }
    return launch_log_probs(a, p->dtype == GEMM_DTYPE_BF16, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

int log_probs_grad(const gemm_log_probs_params *p, const void *logits, const int32_t *tokens, const float *stats,
                   const float *entropy, const float *dlogprob, const float *dentropy, void *dlogits, int64_t ldd,
                   hipStream_t stream)
{
    if (!valid(p) || !valid_ld(ldd, p->vocab)) return GEMM_ERR_INVALID_ARG;
    if (p->rows > 0 && (!logits || !stats || !dlogits || (dlogprob && !tokens) || (dentropy && !entropy)))
        return GEMM_ERR_INVALID_ARG;
    const int es = size_of(p->dtype);
    if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(tokens, 4) || misaligned(stats, 4) ||
        misaligned(entropy, 4) || misaligned(dlogprob, 4) || misaligned(dentropy, 4))
        return GEMM_ERR_INVALID_ARG;
    // in place: a row of the gradient lies over its logits and no others
    if (dlogits == logits && p->rows > 1 && ldd != p->ld) return GEMM_ERR_INVALID_ARG;
    if (p->rows == 0) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    LogProbsGradArgs a{logits, tokens,  stats,   entropy,       dlogprob, dentropy,
                       dlogits, p->ld, ldd, p->rows, (int)p->vocab, p->scale};
    return launch_log_probs_grad(a, p->dtype == GEMM_DTYPE_BF16, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
}

// ---------------------------------------------------- mixture of experts --

constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxRank = 4096;
constexpr int64_t kMaxWeightLd = int64_t(1) << 24;   // byte offsets inside a strip stay below 2^32

int64_t up_columns(const gemm_moe_params &p) { return p.gated ? 2 * p.inner : p.inner; }

bool valid(const gemm_moe_params *p)
{
    if (p == nullptr || !known(p->dtype) || !known(p->dtype_y) ||
        (p->transw != GEMM_OP_N && p->transw != GEMM_OP_T) || p->act < GEMM_ACT_NONE || p->act > GEMM_ACT_SILU ||
        (p->gated != 0 && p->gated != 1))
        return false;
    if (p->tokens < 0 || p->tokens > MOE_MAX_TOKENS || p->hidden < 0 || p->hidden > kMaxWidth || p->inner < 0 ||
        p->inner > kMaxWidth || p->experts < 0 || p->experts > MOE_MAX_EXPERTS || p->top < 0 || p->top > MOE_MAX_TOP)
        return false;
    const bool t = p->transw == GEMM_OP_T;
    const int64_t n = up_columns(*p), up_row = t ? p->hidden : n, up_rows = t ? n : p->hidden;
    const int64_t down_row = t ? p->inner : p->hidden, down_rows = t ? p->hidden : p->inner;
    if (!valid_ld(p->ldx, p->hidden) || !valid_ld(p->ldy, p->hidden) || !valid_ld(p->ldup, up_row) ||
        !valid_ld(p->lddown, down_row) || p->ldup > kMaxWeightLd || p->lddown > kMaxWeightLd)
        return false;
    // the experts' weights do not overlap
    return p->experts <= 1 || up_rows * up_row == 0 || down_rows * down_row == 0 ||
           (p->stride_up >= (up_rows - 1) * p->ldup + up_row && p->stride_down >= (down_rows - 1) * p->lddown + down_row);
}

struct MoeShares {
    MoePlan plan;
    int strips_up, strips_down, max_used, parts;
    int64_t ldh, h_bytes, total;
    bool launchable;
};

MoeShares shares_of(const gemm_moe_params &p)
{
    MoeShares s{};
    const bool t = p.transw == GEMM_OP_T, gated = p.gated != 0;
    const int64_t cus = device_compute_units();
    s.max_used = (int)std::min(p.experts, p.tokens * p.top);
    s.plan.small = p.hidden < 8 || p.inner < 8;
    s.plan.many = p.tokens > 16;
    s.parts = 1;
    auto eights = [](int64_t n) { return ceil_div(n, 8) * 8; };   // xcd_place
    auto strips_up = [&](bool wide) { return ceil_div(p.inner, moe_strip_up(t, gated, wide)); };
    auto strips_down = [&](bool wide) { return ceil_div(p.hidden, moe_strip_down(t, s.plan.many, wide)); };
    // Wide strips where there are blocks for all units four times over.  N x K weights: 1
    // token, 4 experts of 4096 x 2048, 26 us in 512 narrow blocks, 29 in 256 wide ones; 16
    // tokens, 64 of 2048 x 1024, 82 in 4096 narrow ones, 79 in 2048 wide ones.  K x N: 37
    // and 48 us, 114 and 97.  With more tokens narrow strips of N x K weights read too
    // much of x again (20 tokens, 1001 x 2003: 45 us wide, 56 narrow).
    s.plan.wide_up = (t && s.plan.many) || s.max_used * strips_up(true) >= 4 * cus;
    s.strips_up = (int)strips_up(s.plan.wide_up);
    s.plan.blocks_up = eights((int64_t)s.max_used * s.strips_up);
    if (s.plan.small) {
        auto blocks = [&](int64_t width) { return std::min<int64_t>(ceil_div(p.tokens * p.top * width, 256), 65536); };
        s.strips_down = 0;
        s.plan.blocks_up = blocks(p.inner);
        s.plan.blocks_down = blocks(p.hidden);
    } else if (s.plan.many) {
        s.plan.wide_down = t || s.max_used * strips_down(true) >= 4 * cus;
        s.strips_down = (int)strips_down(s.plan.wide_down);
        s.plan.blocks_down = eights((int64_t)s.max_used * s.strips_down);
    } else {
        // Strips and parts by the time that the weights take, at 20 KB per us and unit in
        // wide strips, 17 and 14 in narrow ones of N x K and K x N weights (189 MB, 256
        // units: 40, 47 and 62 us), and 4.5 us for a launch that joins parts.
        const double bytes = (double)s.max_used * (double)p.inner * (double)p.hidden * size_of(p.dtype);
        double best = 0.0;
        for (int wide = 0; wide < 2; ++wide)
            for (int parts = 1; parts <= 8; ++parts) {
                const int64_t blocks = strips_down(wide != 0) * parts;
                if (parts > 1 && (blocks > cus || parts > s.max_used)) break;
                const double rate = wide ? 20e3 : t ? 17e3 : 14e3;
                const double us = bytes / (rate * (double)std::min(cus, blocks)) + (parts > 1 ? 4.5 : 0.0);
                if ((wide == 0 && parts == 1) || us < best) {
                    best = us;
                    s.plan.wide_down = wide != 0;
                    s.parts = parts;
                }
            }
        s.strips_down = (int)strips_down(s.plan.wide_down);
        s.plan.blocks_down = eights((int64_t)s.strips_down * s.parts);
    }
    const int64_t vec = 16 / size_of(p.dtype), places = p.tokens * p.top;
    s.ldh = ceil_div(p.inner, vec) * vec;
    s.h_bytes = (p.dtype == GEMM_DTYPE_BF16 ? 2 : 1) * places * s.ldh * size_of(p.dtype);   // whole 16 bytes
    s.total = s.h_bytes + (s.plan.many || s.plan.small ? places : s.parts > 1 ? s.parts * p.tokens : 0) * p.hidden * 4;
    const int64_t most = int64_t(UINT32_MAX) / 512;   // blocks of a launch
    s.launchable = s.plan.blocks_up <= most && s.plan.blocks_down <= most && p.tokens * ceil_div(p.hidden, 256) <= most;
    return s;
}

int moe_layer(const gemm_moe_params *p, const void *x, const void *up, const void *down, const int32_t *ids,
              const float *weights, const void *residual, void *y, void *workspace, int64_t workspace_bytes,
              hipStream_t stream)
{
    if (!valid(p) || (residual && !valid_ld(p->ldr, p->hidden))) return GEMM_ERR_INVALID_ARG;
    const bool empty = p->tokens == 0 || p->hidden == 0, places = p->top > 0 && p->experts > 0;
    if (!empty && (!y || (places && (!x || !ids || !weights || (p->inner > 0 && (!up || !down))))))
        return GEMM_ERR_INVALID_ARG;
    const int es = size_of(p->dtype);
    if (misaligned(x, es) || misaligned(up, es) || misaligned(down, es) || misaligned(ids, 4) ||
        misaligned(weights, 4) || misaligned(residual, size_of(p->dtype_y)) || misaligned(y, size_of(p->dtype_y)))
        return GEMM_ERR_INVALID_ARG;
    // in place: row r of y lies over row r of the residual and no other
    if (residual && residual == y && p->tokens > 1 && p->ldr != p->ldy) return GEMM_ERR_INVALID_ARG;
    const MoeShares s = shares_of(*p);
    if (!s.launchable || !valid_workspace(workspace, workspace_bytes, empty ? 0 : s.total)) return GEMM_ERR_INVALID_ARG;
    if (empty) return GEMM_OK;
    if (const int rc = need_device()) return rc;
    MoeArgs a{};
    a.x = x;
    a.up = up;
    a.down = down;
    a.ids = ids;
    a.weights = weights;
    a.h = workspace;
    a.h_plane = p->tokens * p->top * s.ldh;
    if (s.total > s.h_bytes) a.ws = reinterpret_cast<float *>(static_cast<char *>(workspace) + s.h_bytes);
    a.e = EpilogueArgs{y, nullptr, residual, nullptr, p->ldy, p->ldr, 0, 1.0f, 1.0f, GEMM_ACT_NONE,
                       p->dtype_y == GEMM_DTYPE_BF16, 0, 0};
    a.ldx = p->ldx;
    a.ldup = p->ldup;
    a.lddown = p->lddown;
    a.ldh = s.ldh;
    a.stride_up = p->experts > 1 ? p->stride_up : 0;
    a.stride_down = p->experts > 1 ? p->stride_down : 0;
    a.tokens = (int)p->tokens;
    a.hidden = (int)p->hidden;
    a.inner = (int)p->inner;
    a.experts = (int)p->experts;
    a.top = places && p->inner > 0 ? (int)p->top : 0;
    a.act = p->act;
    a.gated = p->gated;
    a.strips_up = s.strips_up;
    a.strips_down = s.strips_down;
    a.max_used = s.max_used;
    a.parts = s.parts;
    return launch_moe(a, s.plan, p->dtype == GEMM_DTYPE_BF16, p->transw == GEMM_OP_T, stream) == hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

// ------------------------------------------------------ low-rank adapters --

bool valid(const gemm_adapter_params *p)
{
    if (p == nullptr || !known(p->dtype) || !known(p->dtype_y) || !known(p->dtype_bias) ||
        (p->transw != GEMM_OP_N && p->transw != GEMM_OP_T) || p->act < GEMM_ACT_NONE || p->act > GEMM_ACT_SILU ||
        !in_range(p->rows) || !in_range(p->N) || !in_range(p->K) || !in_range(p->adapters) || p->rank < 0 ||
        p->rank > kMaxRank)
        return false;
    if (!valid_ld(p->lda, p->K) || p->lda > kMaxWeightLd || !valid_ld(p->ldb, p->rank)) return false;
    // the adapters do not overlap
    return p->adapters <= 1 || p->rank == 0 ||
           ((p->K == 0 || p->stride_a >= (p->rank - 1) * p->lda + p->K) &&
            (p->N == 0 || p->stride_b >= (p->N - 1) * p->ldb + p->rank));
}

gemm_linear_params layer_of(const gemm_adapter_params &p)
{
    gemm_linear_params q{};
    q.dtype = p.dtype;
    q.dtype_y = p.dtype_y;
    q.dtype_bias = p.dtype_bias;
    q.transw = p.transw;
    q.act = p.act;
    q.alpha = 1.0f;
    q.rows = p.rows;
    q.N = p.N;
    q.K = p.K;
    q.ldx = p.ldx;
    q.ldw = p.ldw;
    q.ldy = p.ldy;
    q.ldr = p.ldr;
    return q;
}

struct AdapterShares {
    bool any;                  // a row may have an adapter that adds something
    bool join;                 // parts are joined before the product
    int pitch, parts, part_k, slots;
    int64_t t_bytes, ws_bytes, total;    // total < 0: the layer's error
    bool launchable;
};

AdapterShares shares_of(const gemm_adapter_params &p)
{
    AdapterShares s{};
    const gemm_linear_params q = layer_of(p);
    const int64_t layer = gemm_linear_workspace_size(&q);
    s.any = p.rows > 0 && p.N > 0 && p.K > 0 && p.rank > 0 && p.adapters > 0;
    s.launchable = true;
    if (layer < 0) {
        s.total = layer;
        return s;
    }
    s.parts = s.slots = 1;
    s.part_k = (int)p.K;
    s.pitch = (int)(ceil_div(p.rank, 8) * 8);
    if (s.any && p.K >= 8) {
        // A block has 64 rows, a part of K and, of the rows' adapters, every slots-th (blocks
        // behind a group's last adapter end at once).  x and a come to it at 25 KB per us
        // (one row, rank 16, K = 4096: 8.9 us in one part, 5.9 in eight).
        const int64_t groups = ceil_div(p.rows, 64), cus = device_compute_units();
        const int64_t bytes = (std::min<int64_t>(p.rows, 64) + p.rank) * p.K * size_of(p.dtype);
        int64_t want = 1;
        while (want < ADAPTER_MAX_PARTS && bytes / want > 24 * 1024 && 2 * want * groups <= cus && p.K >= 512 * want) want *= 2;
        s.slots = (int)std::max<int64_t>(1, std::min(std::min<int64_t>(p.adapters, std::min<int64_t>(p.rows, 64)),
                                                     2 * cus / (groups * want)));
        s.part_k = (int)(ceil_div(ceil_div(p.K, want), 64) * 64);
        s.parts = (int)ceil_div(p.K, s.part_k);
        s.launchable = groups * s.slots * s.parts <= int64_t(UINT32_MAX) / 512;
    }
    // the sums of a few rows' parts are added up by the product's blocks, if they can
    s.join = s.parts > 1 && (p.rows > 64 || !adapter_sums_allowed(&q));
    const int64_t values = p.rows * s.pitch;       // whole 16 bytes, as bf16 too
    s.ws_bytes = s.any && s.parts > 1 ? s.parts * values * 4 : 0;
    s.t_bytes = s.ws_bytes + (s.any && (s.parts == 1 || s.join) ? values * 4 : 0);   // two bf16 values, or one in fp32
    s.total = s.t_bytes + layer;
    return s;
}

int adapter_linear(const gemm_adapter_params *p, const void *x, const void *w, const void *a, const void *b,
                   const int32_t *ids, const float *scales, const void *bias, const void *residual, void *y,
                   void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    if (!valid(p)) return GEMM_ERR_INVALID_ARG;
    const AdapterShares s = shares_of(*p);
    if (s.total < 0 || !s.launchable || !valid_workspace(workspace, workspace_bytes, s.total)) return GEMM_ERR_INVALID_ARG;
    const int es = size_of(p->dtype);
    if ((s.any && (!x || !a || !b || !ids)) || misaligned(x, es) || misaligned(a, es) || misaligned(b, es) ||
        misaligned(ids, 4) || misaligned(scales, 4))
        return GEMM_ERR_INVALID_ARG;
    const gemm_linear_params q = layer_of(*p);
    char *scratch = static_cast<char *>(workspace);
    void *rest = s.total > s.t_bytes ? scratch + s.t_bytes : nullptr;
    if (!s.any)
        return linear_with_adapters(&q, nullptr, nullptr, x, w, bias, residual, y, rest, s.total - s.t_bytes, stream);
    AdapterDownArgs d{};
    d.x = x;
    d.a = a;
    d.ids = ids;
    d.scales = scales;
    d.ws = static_cast<float *>(workspace);
    d.t = scratch + s.ws_bytes;
    d.join = s.join;
    d.ldx = p->ldx;
    d.lda = p->lda;
    d.stride_a = p->adapters > 1 ? p->stride_a : 0;
    d.plane = p->rows * s.pitch;
    d.rows = (int)p->rows;
    d.K = (int)p->K;
    d.count = (int)p->adapters;
    d.rank = (int)p->rank;
    d.pitch = s.pitch;
    d.parts = s.parts;
    d.part_k = s.part_k;
    d.slots = s.slots;
    AdapterArgs ad{};
    const bool sums = s.parts > 1 && !s.join;
    ad.t = sums ? workspace : d.t;
    ad.parts = sums ? s.parts : 0;
    ad.b = b;
    ad.ids = ids;
    ad.ldb = p->ldb;
    ad.stride_b = p->adapters > 1 ? p->stride_b : 0;
    ad.plane = d.plane;
    ad.count = d.count;
    ad.rank = d.rank;
    ad.pitch = s.pitch;
    return linear_with_adapters(&q, &d, &ad, x, w, bias, residual, y, rest, s.total - s.t_bytes, stream);
}

}  // namespace
}  // namespace dg

extern "C" {

int64_t gemm_moe_layer_workspace_size(const gemm_moe_params *p)
{
    if (!dg::valid(p)) return GEMM_ERR_INVALID_ARG;
    const dg::MoeShares s = dg::shares_of(*p);
    if (!s.launchable) return GEMM_ERR_INVALID_ARG;
    return p->tokens == 0 || p->hidden == 0 ? 0 : s.total;
}

int gemm_moe_layer(const gemm_moe_params *p, const void *x, const void *w_up, const void *w_down, const int32_t *ids,
                   const float *weights, const void *residual, void *y, void *workspace, int64_t workspace_bytes,
                   hipStream_t stream)
{
    return dg::moe_layer(p, x, w_up, w_down, ids, weights, residual, y, workspace, workspace_bytes, stream);
}

int64_t gemm_adapter_linear_workspace_size(const gemm_adapter_params *p)
{
    if (!dg::valid(p)) return GEMM_ERR_INVALID_ARG;
    const dg::AdapterShares s = dg::shares_of(*p);
    return s.launchable ? s.total : GEMM_ERR_INVALID_ARG;
}

int gemm_adapter_linear(const gemm_adapter_params *p, const void *x, const void *w, const void *a, const void *b,
                        const int32_t *ids, const float *scales, const void *bias, const void *residual, void *y,
                        void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    return dg::adapter_linear(p, x, w, a, b, ids, scales, bias, residual, y, workspace, workspace_bytes, stream);
}

int64_t gemm_log_probs_workspace_size(const gemm_log_probs_params *p)
{
    return dg::valid(p) ? dg::log_probs_bytes(*p) : GEMM_ERR_INVALID_ARG;
}

int gemm_log_probs(const gemm_log_probs_params *p, const void *logits, const int32_t *tokens, float *logprob,
                   float *entropy, float *stats, int32_t *top_ids, float *top_logprobs, void *workspace,
                   int64_t workspace_bytes, hipStream_t stream)
{
    return dg::log_probs(p, logits, tokens, logprob, entropy, stats, top_ids, top_logprobs, workspace,
                         workspace_bytes, stream);
}

int gemm_log_probs_grad(const gemm_log_probs_params *p, const void *logits, const int32_t *tokens,
                        const float *stats, const float *entropy, const float *dlogprob, const float *dentropy,
                        void *dlogits, int64_t ldd, hipStream_t stream)
{
    return dg::log_probs_grad(p, logits, tokens, stats, entropy, dlogprob, dentropy, dlogits, ldd, stream);
}

}  // extern "C"
