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
    if (a.stats != nullptr) a.stats[row] = make_float4(0.f, 0.f, 0.f, static_cast<float>(kind));
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

// Results of a good row (x_t, rank: the token's, where there is one). For the backward
// pass: M, 1 / S and the entropy less log S.
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
        a.stats[row] = make_float4(M, 1.0f / S, static_cast<float>(-mean), kRowGood);
    if (a.status != nullptr) a.status[row] = 0;
}

// A row's teacher in shared memory: the tokens that have entries, each once.
struct Teacher {
    int32_t id[SV_MAX_TOP];      // -1 where there is none, or where it came before
    float x[SV_MAX_TOP];         // the student's logit
    float p[SV_MAX_TOP];         // probability (finish_distill renormalises)
    float logp[SV_MAX_TOP];      // as given
    double part[4], part2[4];    // sums of four warps
    float top[4];
    int count[4];
    double mass;                 // the entries' sum, before they are renormalised
    int distinct;
    int status;
    float listed, others;        // what finish_distill leaves: factors of 2^((x - M) c)
};

// Fills in all but x; called by all threads of a block of at least 128. Ends with a
// barrier.
__device__ __forceinline__ void load_teacher(Teacher& t, const DistillArgs& a, int32_t row)
{
    const int j = threadIdx.x;
    if (j == 0) t.status = 0;
    __syncthreads();
    const int warp = j >> 5;
    int32_t id = -1;
    float lp = -inf();
    if (j < SV_MAX_TOP) {
        if (j < a.k) {
            const int64_t at = static_cast<int64_t>(row) * a.k + j;
            id = a.ids[at];
            lp = a.logp[at];
            int bad = 0;
            if (id < -1 || id >= a.r.V) bad = SV_SEQ_BAD_TOKEN;
            if (lp != lp || lp == inf()) bad |= SV_SEQ_NONFINITE;
            if (bad != 0) {
                atomicOr(&t.status, bad);
                id = -1;
            }
            if (id < 0) lp = -inf();
        }
        t.id[j] = id;
        t.logp[j] = lp;
        float top = lp;
        for (int off = 16; off > 0; off >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
        if ((j & 31) == 0) t.top[warp] = top;
    }
    __syncthreads();
    if (j < SV_MAX_TOP) {
        // Renormalised probabilities are taken from the largest one, so that none
        // overflows.
        float shift = 0.f;
        if (!a.bucket) {
            shift = fmaxf(fmaxf(t.top[0], t.top[1]), fmaxf(t.top[2], t.top[3]));
            if (shift == -inf()) shift = 0.f;
        }
        bool first = id >= 0;
        float p = 0.f;
        for (int i = 0; i < a.k; ++i)
            if (t.id[i] == id) {
                if (i < j) first = false;
                p += expf(t.logp[i] - shift);
            }
        if (!first) p = 0.f;
        double sum = p;
        int n = first;
        for (int off = 16; off > 0; off >>= 1) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
        }
        if ((j & 31) == 0) {
            t.part[warp] = sum;
            t.count[warp] = n;
        }
        t.p[j] = p;
        id = first ? id : -1;
    }
    __syncthreads();
    if (j < SV_MAX_TOP) t.id[j] = id;
    if (j == 0) {
        t.mass = (t.part[0] + t.part[1]) + (t.part[2] + t.part[3]);
        t.distinct = (t.count[0] + t.count[1]) + (t.count[2] + t.count[3]);
        if (!a.bucket && t.distinct > 0 && !(t.mass > 0.0)) t.status |= SV_SEQ_NONFINITE;
    }
    __syncthreads();
}

// Loss and gradient factors of a good row, from M, the largest logit, and the sum S_o of
// 2^((x - M) c) over the tokens without entries; the entries' logits are in t.x. The
// gradient is then, times the row's weight over T,
//   listed 2^((x - M) c) - p   for tokens with entries,   others 2^((x - M) c)   for others:
// with S the sum over all tokens and m the entries' probabilities' sum,
//   listed = 1 / S, others = 1 / S                          renormalised
//   listed = max(m, 1) / S                                  bucket
//   others = (1 - P_o / q_o) / S = (m - q_e) / S_o          .. where m <= 1 (q_e = 1 - q_o)
// Called by all threads; ends with a barrier.
__device__ __forceinline__ void finish_distill(Teacher& t, const DistillArgs& a, int32_t row,
                                               float M, float S_o)
{
    const int j = threadIdx.x, warp = j >> 5;
    float e = 0.f;
    if (j < SV_MAX_TOP) {
        if (t.id[j] >= 0) e = ex2((t.x[j] - M) * a.r.c);
        double sum = e;
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        if ((j & 31) == 0) t.part[warp] = sum;
    }
    __syncthreads();
    const double S_e = (t.part[0] + t.part[1]) + (t.part[2] + t.part[3]);
    const double S = S_e + S_o;
    const bool has_others = t.distinct < a.r.V;
    if (j < SV_MAX_TOP) {
        const double log_s = log_wide(static_cast<float>(S));
        double term = 0.0;
        const float p = t.p[j];
        if (t.id[j] >= 0 && p > 0.f) {
            const double log_m = a.bucket ? 0.0 : log_wide(static_cast<float>(t.mass));
            const double P = a.bucket ? p : p / t.mass;
            term = P * (log_wide(p) - log_m - log_prob(t.x[j], M, a.r.c, log_s));
            t.p[j] = static_cast<float>(P);
        }
        for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, off);
        if ((j & 31) == 0) t.part2[warp] = term;
    }
    __syncthreads();
    if (j == 0) {
        double loss = (t.part2[0] + t.part2[1]) + (t.part2[2] + t.part2[3]);
        const float m = static_cast<float>(t.mass);
        const float q_e = static_cast<float>(S_e / S);
        t.listed = t.others = static_cast<float>(1.0 / S);
        if (a.bucket) {
            const double P_o = has_others ? fmax(0.0, 1.0 - t.mass) : 0.0;
            if (P_o > 0.0) {
                const double log_P = m < 0.5f ? log1pf(-m) : logf(static_cast<float>(P_o));
                const double log_q = q_e < 0.5f ? static_cast<double>(log1pf(-q_e))
                                                : log_wide(S_o) - log_wide(static_cast<float>(S));
                loss += P_o * (log_P - log_q);
            }
            const double total = t.mass + P_o;
            t.listed = static_cast<float>(total / S);
            // (no token left, or all of probability 0: their gradient is 0)
            t.others = !(S_o > 0.f)   ? 0.f
                       : t.mass <= 1.0 ? static_cast<float>((t.mass - S_e / S) / S_o)
                                       : t.listed;
        }
        if (a.loss != nullptr) a.loss[row] = static_cast<float>(loss);
        if (a.stats != nullptr) a.stats[row] = make_float4(M, t.listed, t.others, kRowGood);
        if (a.status != nullptr) a.status[row] = 0;
    }
    __syncthreads();
}

// The same for a row without entries, or a bad one.
__device__ __forceinline__ void finish_distill_plain(const DistillArgs& a, int32_t row, int kind,
                                                     int status)
{
    if (a.loss != nullptr) a.loss[row] = kind == kRowBad ? nan() : 0.f;
    if (a.stats != nullptr) a.stats[row] = make_float4(0.f, 0.f, 0.f, static_cast<float>(kind));
    if (a.status != nullptr) a.status[row] = status;
}

}  // namespace svl
