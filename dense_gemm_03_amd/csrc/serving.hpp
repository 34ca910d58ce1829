// Arguments and launchers of the operators of gemm_serving.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_linear.h"
#include "linear_kernel.hpp"

namespace dg {

struct LogProbsArgs {
    const void *logits;
    const int32_t *tokens;       // or nullptr
    float *logprob, *entropy, *stats, *top_logprobs;   // each may be nullptr
    int32_t *top_ids;
    int64_t ld;
    int64_t rows;
    int vocab, top;
    float scale;
    // of a row: `parts` parts of `part_chunks` chunks, each by a team of `team`
    // waves; with more than one part, their sums and lists meet in ws
    int parts, part_chunks, team;
    float *ws;                   // per row and part: m, s, u, -
    uint64_t *ws_keys;           // and `top` keys
};
hipError_t launch_log_probs(const LogProbsArgs &args, bool bf16, hipStream_t stream);
// Logits per chunk, the least that a wave takes.
int log_probs_chunk();

struct LogProbsGradArgs {
    const void *logits;
    const int32_t *tokens;
    const float *stats, *entropy, *dlogprob, *dentropy;
    void *dlogits;
    int64_t ld, ldd;
    int64_t rows;
    int vocab;
    float scale;
};
hipError_t launch_log_probs_grad(const LogProbsGradArgs &args, bool bf16, hipStream_t stream);

constexpr int MOE_MAX_TOP = 32;
constexpr int MOE_MAX_EXPERTS = 1024;
constexpr int MOE_MAX_TOKENS = 512;

struct MoeArgs {
    const void *x, *up, *down;
    const int32_t *ids;
    const float *weights;
    void *h;                     // the first product's results: a row of ldh per place (token, j)
    int64_t h_plane;             // elements from h's upper halves to its lower ones (bf16)
    float *ws;                   // y of `parts` > 1 parts; with many tokens, the rows of all places
    EpilogueArgs e;
    int64_t ldx, ldup, lddown, ldh, stride_up, stride_down;
    int tokens, hidden, inner, experts, top, act, gated;
    int strips_up, strips_down;
    int max_used;                // experts that the tokens can name
    int parts;                   // of the second product's sum
};
struct MoePlan {
    bool small;                  // a width below 8: a thread per value
    bool many;                   // more than 16 tokens
    bool wide_up, wide_down;     // strips of a block
    int64_t blocks_up, blocks_down;
};
// Columns of a block of the first product, and of the second.
int moe_strip_up(bool transw, bool gated, bool wide);
int moe_strip_down(bool transw, bool many, bool wide);
hipError_t launch_moe(const MoeArgs &args, const MoePlan &plan, bool bf16, bool transw, hipStream_t stream);

// t = scale x . a^T of each row's adapter, as AdapterArgs has it.
struct AdapterDownArgs {
    const void *x, *a;           // a: per adapter rank x K
    const int32_t *ids;
    const float *scales;         // or nullptr: 1
    void *t;
    float *ws;                   // sums of more than one part: parts x rows x pitch
    int64_t ldx, lda, stride_a, plane;
    int rows, K, count, rank, pitch;
    int parts, part_k;           // parts of K, of part_k values
    int join;                    // whether to form t of more than one part, or leave the sums
    int slots;                   // blocks per 64 rows and part: each takes every slots-th adapter of the rows
};
hipError_t launch_adapter_down(const AdapterDownArgs &args, bool bf16, hipStream_t stream);

// Whether the kernel that this layer takes can add up the adapters' sums of parts.
bool adapter_sums_allowed(const gemm_linear_params *p);

// gemm_linear with an adapter per row (linear_api.hip): launch_adapter_down(*down) once
// the arguments are checked, then the layer with *ad.  Both nullptr: the layer alone.
// Returns a gemm_status.
int linear_with_adapters(const gemm_linear_params *p, const AdapterDownArgs *down, const AdapterArgs *ad,
                         const void *x, const void *w, const void *bias, const void *residual, void *y,
                         void *workspace, int64_t workspace_bytes, hipStream_t stream);

}  // namespace dg
