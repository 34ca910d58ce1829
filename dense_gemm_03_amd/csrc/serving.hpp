// Arguments and launchers of the operators of gemm_serving.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

}  // namespace dg
