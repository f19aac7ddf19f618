// lp_internal.h -- launchers of libsvlogprobs' translation units.
#pragma once

#include "lp_common.cuh"

namespace svl {

// What the backward pass is told of a row (SV_ROW_STATS floats).
enum RowKind { kRowGood = 0, kRowSkipped = 1, kRowBad = 2 };
struct __align__(16) RowStats {
    float M;           // the largest logit; distillation: of the tokens without entries
    float scale;       // factor of 2^((x - M) c)
    float mean;        // log probabilities: entropy less log S
    float listed_M;    // distillation: the largest logit of all,
    float listed;      //   the factor of 2^((x - listed_M) c) for tokens with entries,
    float shift, inv;  //   and their probabilities: exp(log probability - shift) inv
    float kind;
};

struct LogprobArgs {
    Rows r;
    const int32_t* tokens;
    int32_t k;
    float* logprobs;
    float* entropy;
    float* lse;
    int32_t* rank;
    int32_t* top_tokens;
    float* top_logprobs;
    RowStats* stats;
    int32_t* status;
};

struct LogprobGradArgs {
    Rows r;
    const int32_t* tokens;
    const RowStats* stats;
    const float* a;  // gradients of log probability, entropy and lse
    const float* b;
    const float* c;
    RowAt grad;
};

struct DistillArgs {
    Rows r;
    const int32_t* ids;
    const float* logp;
    int32_t k;
    int32_t bucket;
    const float* weights;
    float* loss;
    RowAt grad;       // base NULL: no gradient
    RowStats* stats;
    int32_t* status;
};

// (bytes of workspace, 0: none is used)
size_t logprobs_workspace(const Rows& r, int dtype, int32_t k);
size_t distill_workspace(const Rows& r, int dtype);
cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, void* workspace, cudaStream_t s);
cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, int dtype, cudaStream_t s);
// (all_done: false if the gradient that is asked for has still to be launched)
cudaError_t launch_distill(const DistillArgs& a, int dtype, void* workspace, bool* all_done,
                           cudaStream_t s);
// (a.weights: the loss's gradient, NULL for ones; behind: launch_distill is just before it in the
// stream)
cudaError_t launch_distill_grad(const DistillArgs& a, int dtype, bool behind, cudaStream_t s);

}  // namespace svl
