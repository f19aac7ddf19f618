// lp_finish.cuh -- the end of a row: results from its maximum and sums.
//
// Sums are relative to the row's largest logit M: S = sum 2^((x - M) c),
// E = sum 2^((x - M) c) (x - M) c, with c = log2(e) / T. The differences x - M of
// 16-bit logits are exact where they matter, whatever the size of the logits. All of
// a row's numbers use the same float c, so that its rounding is one of the
// temperature (2^-24 of it) and never a difference between two logarithms. The few
// logarithms of a row are combined in 64 bits: a divergence is a small difference of
// numbers near 10, which 32 bits would round at 10^-6.
#pragma once

#include "lp_internal.h"

namespace svl {

// log of 2^((x - M) c) / S.
__device__ __forceinline__ double log_prob(float x, float M, float c, double log_s)
{
    return (static_cast<double>(x) - M) * c * 0.693147180559945309417 - log_s;
}

// Results of a row of which nothing is asked, or which is bad.
__device__ __forceinline__ void finish_plain(const LogprobArgs& a, int32_t row, int kind,
                                             int status)
{
    const float f = kind == kRowBad ? nan() : 0.f;
    if (a.logprobs != nullptr) a.logprobs[row] = f;
    if (a.entropy != nullptr) a.entropy[row] = f;
    if (a.lse != nullptr) a.lse[row] = f;
    if (a.rank != nullptr) a.rank[row] = -1;
    if (a.stats != nullptr) a.stats[row].kind = kind;
    if (a.status != nullptr) a.status[row] = status;
}

__device__ __forceinline__ void finish_plain_top(const LogprobArgs& a, int32_t row, int kind,
                                                 int tid, int threads)
{
    for (int j = tid; j < a.k; j += threads) {
        a.top_tokens[static_cast<int64_t>(row) * a.k + j] = -1;
        a.top_logprobs[static_cast<int64_t>(row) * a.k + j] = kind == kRowBad ? nan() : -inf();
    }
}

// Results of a good row (x_t, rank: the token's, where there is one).
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int32_t row, float M, float S,
                                           float E, float x_t, int rank, double log_s)
{
    const double mean = static_cast<double>(E / S) * 0.693147180559945309417;  // of log p S
    if (a.logprobs != nullptr)
        a.logprobs[row] = static_cast<float>(log_prob(x_t, M, a.r.c, log_s));
    if (a.rank != nullptr) a.rank[row] = rank;
    if (a.entropy != nullptr) a.entropy[row] = static_cast<float>(log_s - mean);
    if (a.lse != nullptr)
        a.lse[row] = static_cast<float>(static_cast<double>(M) * a.r.inv_t + log_s);
    if (a.stats != nullptr)
        a.stats[row] = {M, 1.0f / S, static_cast<float>(-mean), 0.f, 0.f, 0.f, 0.f, kRowGood};
    if (a.status != nullptr) a.status[row] = 0;
}

}  // namespace svl
