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
#include "lp_vec.cuh"

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

// A row's teacher in shared memory: the tokens that have entries, each once.
constexpr int kChunks = SV_MAX_TOP / 32;
struct Teacher {
    int32_t id[SV_MAX_TOP];      // -1 where there is none, or where it came before
    float x[SV_MAX_TOP];         // the student's logit
    float p[SV_MAX_TOP];         // probability (finish_distill renormalises)
    float logp[SV_MAX_TOP];      // as given
    double part[kChunks], part2[kChunks];  // sums of 32 entries
    float top[kChunks];
    int count[kChunks];
    double mass;                 // the entries' sum, before they are renormalised
    float shift;                 // what was taken off their log probabilities
    int distinct;
    int status;
    // What finish_distill leaves: the gradient is, times the row's weight over T,
    //   scale 2^((x - M) c)                for tokens without entries
    //   listed 2^((x - listed_M) c) - p    for tokens with
    float M, scale, listed_M, listed;
};

// Sum of the 32 lanes of a warp.
template <typename N>
__device__ __forceinline__ N warp_sum(N x)
{
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    return x;
}

// Sum over the chunks in use, in one order.
template <typename N>
__device__ __forceinline__ N chunk_sum(const N* part, int chunks)
{
    N s = part[0];
    for (int i = 1; i < chunks; ++i) s += part[i];
    return s;
}

// Takes the row's entries and says whether there is anything to do with it (an entry, or a
// fault); called by all threads, with a barrier inside and at its end.
__device__ __forceinline__ bool read_teacher(Teacher& t, const DistillArgs& a, int32_t row)
{
    int any = 0;
    for (int j = threadIdx.x; j < SV_MAX_TOP; j += blockDim.x) {
        int32_t id = -1;
        float lp = -inf();
        if (j < a.k) {
            const int64_t at = static_cast<int64_t>(row) * a.k + j;
            id = a.ids[at];
            lp = a.logp[at];
        }
        any |= id != -1 || lp != lp || lp == inf();
        t.id[j] = id;
        t.logp[j] = lp;
    }
    if (threadIdx.x == 0) t.status = 0;
    return __syncthreads_or(any) != 0;
}

// The rest of the teacher but the student's logits, after read_teacher. Ends with a barrier.
__device__ __forceinline__ void make_teacher(Teacher& t, const DistillArgs& a)
{
    const int end = (a.k + 31) & ~31, chunks = end >> 5;
    for (int j = threadIdx.x; j < end; j += blockDim.x) {
        int32_t id = t.id[j];
        float lp = t.logp[j];
        int bad = 0;
        if (id < -1 || id >= a.r.V) bad = SV_SEQ_BAD_TOKEN;
        if (lp != lp || lp == inf()) bad |= SV_SEQ_NONFINITE;
        if (bad != 0) {
            atomicOr(&t.status, bad);
            id = -1;
        }
        if (id < 0) lp = -inf();
        t.id[j] = id;
        t.logp[j] = lp;
        const float top = warp_max(lp);
        if ((j & 31) == 0) t.top[j >> 5] = top;
    }
    __syncthreads();
    // Renormalised probabilities are taken from the largest one, so that none overflows.
    float shift = 0.f;
    if (!a.bucket) {
        shift = t.top[0];
        for (int i = 1; i < chunks; ++i) shift = fmaxf(shift, t.top[i]);
        if (shift == -inf()) shift = 0.f;
    }
    uint32_t again = 0;  // (entries of this thread whose token came before)
    int turn = 0;
    for (int j = threadIdx.x; j < end; j += blockDim.x, ++turn) {
        const int32_t id = t.id[j];
        bool first = id >= 0;
        float p = 0.f;
        if (id >= 0)
            for (int i = 0; i < a.k; ++i)
                if (t.id[i] == id) {
                    if (i < j) first = false;
                    p += expf(t.logp[i] - shift);
                }
        if (!first) {
            p = 0.f;
            again |= 1u << turn;
        }
        const double sum = warp_sum(static_cast<double>(p));
        const int n = warp_sum(first ? 1 : 0);
        if ((j & 31) == 0) {
            t.part[j >> 5] = sum;
            t.count[j >> 5] = n;
        }
        t.p[j] = p;
    }
    __syncthreads();
    turn = 0;
    for (int j = threadIdx.x; j < end; j += blockDim.x, ++turn)
        if (again >> turn & 1) t.id[j] = -1;
    if (threadIdx.x == 0) {
        t.shift = shift;
        t.mass = chunk_sum(t.part, chunks);
        t.distinct = chunk_sum(t.count, chunks);
        if (!a.bucket && t.distinct > 0 && !(t.mass > 0.0)) t.status |= SV_SEQ_NONFINITE;
    }
    __syncthreads();
}

// Loss and gradient factors of a row, from the largest logit M_o and the sum S_o of
// 2^((x - M_o) c) over the tokens without entries (-inf and 0: none, or all of them are
// -inf); the entries' logits are in t.x. With M the largest of all, S the sum over all of
// 2^((x - M) c), q_e the entries' share of it and m the sum of their probabilities:
//   listed = 1 / S, scale = 2^((M_o - M) c) / S             renormalised
//   listed = max(m, 1) / S                                  bucket
//   scale  = (1 - P_o / q_o) 2^((M_o - M) c) / S = (m - q_e) / S_o     .. where m <= 1
// so that the others' gradient keeps its digits however small their share is. Called by
// all threads; `lead` writes the results. Returns the row's kind; ends with a barrier.
__device__ __forceinline__ int finish_distill(Teacher& t, const DistillArgs& a, int32_t row,
                                              float M_o, float S_o, bool lead)
{
    const int end = (a.k + 31) & ~31, chunks = end >> 5;
    const float c = a.r.c;
    for (int j = threadIdx.x; j < end; j += blockDim.x) {
        const float top = warp_max(t.id[j] >= 0 ? t.x[j] : -inf());
        if ((j & 31) == 0) t.top[j >> 5] = top;
    }
    __syncthreads();
    float M = M_o;
    for (int i = 0; i < chunks; ++i) M = fmax_nan(M, t.top[i]);
    const bool good = fabsf(M) < inf() && t.status == 0;
    if (!good) {
        if (lead && threadIdx.x == 0) {
            const int status = t.status | (fabsf(M) < inf() ? 0 : SV_SEQ_NONFINITE);
            if (a.loss != nullptr) a.loss[row] = nan();
            if (a.stats != nullptr) a.stats[row].kind = kRowBad;
            if (a.status != nullptr) a.status[row] = status;
        }
        return kRowBad;
    }
    for (int j = threadIdx.x; j < end; j += blockDim.x) {
        const float e = t.id[j] >= 0 ? ex2((t.x[j] - M) * c) : 0.f;
        const double sum = warp_sum(static_cast<double>(e));
        if ((j & 31) == 0) t.part[j >> 5] = sum;
    }
    __syncthreads();
    const float fall = S_o > 0.f ? ex2((M_o - M) * c) : 0.f;
    const double S_e = chunk_sum(t.part, chunks);
    const double S = S_e + static_cast<double>(S_o) * fall;
    const double log_s = log_wide(static_cast<float>(S));
    for (int j = threadIdx.x; j < end; j += blockDim.x) {
        double term = 0.0;
        const float p = t.p[j];
        if (t.id[j] >= 0 && p > 0.f) {
            const double log_m = a.bucket ? 0.0 : log_wide(static_cast<float>(t.mass));
            const double P = a.bucket ? p : p / t.mass;
            term = P * (log_wide(p) - log_m - log_prob(t.x[j], M, c, log_s));
            t.p[j] = static_cast<float>(P);
        }
        term = warp_sum(term);
        if ((j & 31) == 0) t.part2[j >> 5] = term;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double loss = chunk_sum(t.part2, chunks);
        const double q_e = S_e / S;
        t.M = S_o > 0.f ? M_o : 0.f;  // (nothing finite: any finite number)
        t.listed_M = M;
        t.listed = static_cast<float>(1.0 / S);
        t.scale = t.listed * fall;
        if (a.bucket) {
            const double P_o = t.distinct < a.r.V ? fmax(0.0, 1.0 - t.mass) : 0.0;
            if (P_o > 0.0) {
                const float m = static_cast<float>(t.mass);
                const double log_P = m < 0.5f ? log1pf(-m) : logf(static_cast<float>(P_o));
                const double log_q = q_e < 0.5 ? static_cast<double>(log1pf(-static_cast<float>(q_e)))
                                               : log_prob(M_o, M, c, log_s) + log_wide(S_o);
                loss += P_o * (log_P - log_q);
            }
            t.listed = static_cast<float>((t.mass + P_o) / S);
            // (no other token, or all of probability 0: their gradient is 0)
            t.scale = !(S_o > 0.f)    ? 0.f
                      : t.mass <= 1.0 ? static_cast<float>((t.mass - q_e) / S_o)
                                      : t.listed * fall;
        }
        if (lead) {
            if (a.loss != nullptr) a.loss[row] = static_cast<float>(loss);
            if (a.stats != nullptr)
                a.stats[row] = {t.M,     t.scale,
                                0.f,     t.listed_M,
                                t.listed, t.shift,
                                a.bucket ? 1.f : static_cast<float>(1.0 / t.mass),
                                kRowGood};
            if (a.status != nullptr) a.status[row] = 0;
        }
    }
    __syncthreads();
    return kRowGood;
}

// The same for a row without entries.
__device__ __forceinline__ void finish_distill_skipped(const DistillArgs& a, int32_t row)
{
    if (a.loss != nullptr) a.loss[row] = 0.f;
    if (a.stats != nullptr) a.stats[row].kind = kRowSkipped;
    if (a.status != nullptr) a.status[row] = 0;
}

}  // namespace svl
