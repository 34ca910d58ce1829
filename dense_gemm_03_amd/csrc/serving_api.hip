// C ABI of gemm_serving.h: argument checks, choice of variants, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "gemm_internal.hpp"
#include "gemm_serving.h"
#include "serving.hpp"

namespace dg {
namespace {

constexpr int64_t kMaxSize = int64_t(1) << 30;   // as gemm.h
constexpr int64_t kMaxLd = int64_t(1) << 40;

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
           p->top >= 0 && p->top <= 64 && p->top <= p->vocab && std::isfinite(p->scale) && p->scale > 0.0f &&
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

}  // namespace
}  // namespace dg

extern "C" {

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
