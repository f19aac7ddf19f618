// lp_api.cu -- the C ABI (include/sv_logprobs.h): argument checks and launches.
#include <cmath>

#include "lp_internal.h"
#include "lp_stream.cuh"

#define SV_EXPORT extern "C" __attribute__((visibility("default")))

static_assert(svl::kMaxSplitRows * 4 == SV_LOGPROBS_COUNTER_BYTES, "as the header says");
static_assert(sizeof(svl::RowStats) == SV_ROW_STATS * sizeof(float), "as the header says");

namespace {

constexpr int64_t kMax31 = int64_t(1) << 31;
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int element_size(int dtype) { return dtype == SV_F32 ? 4 : 2; }

// Host checks of a description of rows, and the kernels' form of it.
int check_rows(const sv_logit_rows* d, svl::Rows* r, bool pointers = true)
{
    if (d == nullptr) return SV_ERR_ARG;
    if (d->dtype != SV_F32 && d->dtype != SV_BF16 && d->dtype != SV_F16) return SV_ERR_DTYPE;
    if (d->outer < 0 || d->inner < 0 || d->vocab < 1) return SV_ERR_ARG;
    if (d->vocab >= kMax31 || d->outer >= kMax31 || d->inner >= kMax31 ||
        d->outer * d->inner >= kMax31)
        return SV_ERR_SIZE;
    const float T = d->temperature;
    const double c = 1.44269504088896340736 / T;
    // (up to 2^117 two logits that float32 cannot subtract are 2^128 c > 2900 bits apart at least, and
    // the lower one's weight is 0 whether their difference is infinite or not)
    if (!(T > 0.f) || !(T <= 0x1p117f) || !std::isfinite(static_cast<float>(c)) ||
        !std::isfinite(1.0f / T))
        return SV_ERR_ARG;
    const int64_t rows = d->outer * d->inner;
    const int es = element_size(d->dtype);
    const int64_t so = d->outer <= 1 || !pointers ? 0 : d->outer_stride;
    const int64_t si = d->inner <= 1 || !pointers ? 0 : d->inner_stride;
    if (so < 0 || si < 0 || so > kMaxStride || si > kMaxStride) return SV_ERR_ARG;
    if (pointers && rows > 0 && d->logits == nullptr) return SV_ERR_ARG;
    if (pointers && !aligned(d->logits, es)) return SV_ERR_ALIGN;
    r->x = {static_cast<uint8_t*>(const_cast<void*>(d->logits)), so * es, si * es};
    r->inner = static_cast<int32_t>(d->inner > 0 ? d->inner : 1);
    r->rows = static_cast<int32_t>(rows);
    r->V = static_cast<int32_t>(d->vocab);
    r->c = static_cast<float>(c);
    r->inv_t = 1.0f / T;
    return SV_OK;
}

// The gradient's rows; they must not overlap.
int check_grad(const sv_logit_rows* d, void* grad, int64_t so, int64_t si, svl::RowAt* out)
{
    const int es = element_size(d->dtype);
    const int64_t no = d->outer, ni = d->inner, V = d->vocab;
    if (no <= 1) so = 0;
    if (ni <= 1) si = 0;
    if (so < 0 || si < 0 || so > kMaxStride || si > kMaxStride) return SV_ERR_ARG;
    if (no * ni > 0) {
        if (grad == nullptr) return SV_ERR_ARG;
        if ((no > 1 && so < V) || (ni > 1 && si < V)) return SV_ERR_ARG;
        // (sizes are below 2^31 and strides up to 2^40, so (n - 1) stride may pass 2^63)
        const auto apart = [V](int64_t step, int64_t n, int64_t stride) {
            return static_cast<double>(step) >=
                   static_cast<double>(n - 1) * static_cast<double>(stride) + V;
        };
        if (no > 1 && ni > 1 && !apart(so, ni, si) && !apart(si, no, so)) return SV_ERR_ARG;
    }
    if (!aligned(grad, es)) return SV_ERR_ALIGN;
    *out = {static_cast<uint8_t*>(grad), so * es, si * es};
    return SV_OK;
}

int check_teacher(const svl::Rows& r, const int32_t* ids, const float* logp, int64_t k, int tail)
{
    if (k < 1 || (tail != SV_TAIL_RENORMALISE && tail != SV_TAIL_BUCKET)) return SV_ERR_ARG;
    if (k > SV_MAX_TOP) return SV_ERR_SIZE;
    if (r.rows > 0 && (ids == nullptr || logp == nullptr)) return SV_ERR_ARG;
    return aligned(ids, 4) && aligned(logp, 4) ? SV_OK : SV_ERR_ALIGN;
}

size_t up(size_t n) { return (n + 255) & ~size_t(255); }

bool enough(const void* workspace, size_t bytes, size_t need)
{
    return need == 0 || (workspace != nullptr && bytes >= need && aligned(workspace, 256));
}

// Where in a workspace the rows' statistics are: behind the pieces', and the counters in any
// case, which other calls find 0.
size_t stats_offset(const svl::Rows& r, int dtype)
{
    const size_t pieces = svl::distill_workspace(r, dtype);
    return up(pieces > SV_LOGPROBS_COUNTER_BYTES ? pieces : SV_LOGPROBS_COUNTER_BYTES);
}

size_t distill_bytes(const svl::Rows& r, int dtype, bool grad)
{
    return grad ? stats_offset(r, dtype) + static_cast<size_t>(r.rows) * sizeof(svl::RowStats)
                : svl::distill_workspace(r, dtype);
}

int done(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

}  // namespace

SV_EXPORT int sv_logprobs_workspace_bytes(const sv_logit_rows* rows, int64_t top_k, size_t* bytes)
{
    svl::Rows r;
    const int rc = check_rows(rows, &r, false);
    if (rc != SV_OK) return rc;
    if (bytes == nullptr || top_k < 0 || top_k > r.V) return SV_ERR_ARG;
    if (top_k > SV_MAX_TOP || (top_k > 0 && r.V > SV_MAX_TOP_VOCAB)) return SV_ERR_SIZE;
    // (calls with fewer alternatives, or none, may cut rows into more pieces)
    size_t most = distill_bytes(r, rows->dtype, true);
    for (const int64_t k : {top_k, int64_t(0)}) {
        const size_t n = svl::logprobs_workspace(r, rows->dtype, static_cast<int32_t>(k));
        most = n > most ? n : most;
    }
    *bytes = most;
    return SV_OK;
}

SV_EXPORT int sv_token_logprobs(const sv_logit_rows* rows, const int32_t* tokens, int64_t top_k,
                                float* logprobs, float* entropy, float* lse, int32_t* rank,
                                int32_t* top_tokens, float* top_logprobs, float* row_stats,
                                int32_t* row_status, void* workspace, size_t workspace_bytes,
                                void* stream)
{
    svl::LogprobArgs a{};
    const int rc = check_rows(rows, &a.r);
    if (rc != SV_OK) return rc;
    if (top_k < 0 || top_k > a.r.V) return SV_ERR_ARG;
    if (top_k > SV_MAX_TOP || (top_k > 0 && a.r.V > SV_MAX_TOP_VOCAB)) return SV_ERR_SIZE;
    if (tokens == nullptr && (logprobs != nullptr || rank != nullptr) && a.r.rows > 0)
        return SV_ERR_ARG;
    if ((top_tokens == nullptr) != (top_logprobs == nullptr)) return SV_ERR_ARG;
    if (top_k > 0 && top_tokens == nullptr && a.r.rows > 0) return SV_ERR_ARG;
    for (const void* p : {static_cast<const void*>(tokens), static_cast<const void*>(logprobs),
                          static_cast<const void*>(entropy), static_cast<const void*>(lse),
                          static_cast<const void*>(rank), static_cast<const void*>(top_tokens),
                          static_cast<const void*>(top_logprobs),
                          static_cast<const void*>(row_status)})
        if (!aligned(p, 4)) return SV_ERR_ALIGN;
    if (!aligned(row_stats, 16)) return SV_ERR_ALIGN;
    if (a.r.rows == 0) return SV_OK;
    if (!enough(workspace, workspace_bytes,
                svl::logprobs_workspace(a.r, rows->dtype, static_cast<int32_t>(top_k))))
        return SV_ERR_WORKSPACE;
    a.tokens = tokens;
    a.k = static_cast<int32_t>(top_k);
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.lse = lse;
    a.rank = rank;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    a.stats = reinterpret_cast<svl::RowStats*>(row_stats);
    a.status = row_status;
    return done(svl::launch_logprobs(a, rows->dtype, workspace, static_cast<cudaStream_t>(stream)));
}

SV_EXPORT int sv_token_logprobs_backward(const sv_logit_rows* rows, const int32_t* tokens,
                                         const float* row_stats, const float* grad_logprobs,
                                         const float* grad_entropy, const float* grad_lse,
                                         void* grad, int64_t grad_outer_stride,
                                         int64_t grad_inner_stride, void* stream)
{
    svl::LogprobGradArgs a{};
    int rc = check_rows(rows, &a.r);
    if (rc != SV_OK) return rc;
    rc = check_grad(rows, grad, grad_outer_stride, grad_inner_stride, &a.grad);
    if (rc != SV_OK) return rc;
    if (a.r.rows > 0 && (row_stats == nullptr || (tokens == nullptr && grad_logprobs != nullptr)))
        return SV_ERR_ARG;
    if (!aligned(row_stats, 16) || !aligned(tokens, 4) || !aligned(grad_logprobs, 4) ||
        !aligned(grad_entropy, 4) || !aligned(grad_lse, 4))
        return SV_ERR_ALIGN;
    if (a.r.rows == 0) return SV_OK;
    a.tokens = tokens;
    a.stats = reinterpret_cast<const svl::RowStats*>(row_stats);
    a.a = grad_logprobs;
    a.b = grad_entropy;
    a.c = grad_lse;
    return done(svl::launch_logprobs_grad(a, rows->dtype, static_cast<cudaStream_t>(stream)));
}

SV_EXPORT int sv_distill(const sv_logit_rows* rows, const int32_t* teacher_tokens,
                         const float* teacher_logprobs, int64_t k, int tail, const float* weights,
                         float* loss, void* grad, int64_t grad_outer_stride,
                         int64_t grad_inner_stride, float* row_stats, int32_t* row_status,
                         void* workspace, size_t workspace_bytes, void* stream)
{
    svl::DistillArgs a{};
    int rc = check_rows(rows, &a.r);
    if (rc == SV_OK) rc = check_teacher(a.r, teacher_tokens, teacher_logprobs, k, tail);
    if (rc == SV_OK && grad != nullptr)
        rc = check_grad(rows, grad, grad_outer_stride, grad_inner_stride, &a.grad);
    if (rc != SV_OK) return rc;
    if (!aligned(weights, 4) || !aligned(loss, 4) || !aligned(row_stats, 16) ||
        !aligned(row_status, 4))
        return SV_ERR_ALIGN;
    if (a.r.rows == 0) return SV_OK;
    a.ids = teacher_tokens;
    a.logp = teacher_logprobs;
    a.k = static_cast<int32_t>(k);
    a.bucket = tail == SV_TAIL_BUCKET;
    a.weights = weights;
    a.loss = loss;
    a.stats = reinterpret_cast<svl::RowStats*>(row_stats);
    a.status = row_status;
    if (!enough(workspace, workspace_bytes, distill_bytes(a.r, rows->dtype, grad != nullptr)))
        return SV_ERR_WORKSPACE;
    if (grad != nullptr && row_stats == nullptr)
        a.stats = reinterpret_cast<svl::RowStats*>(static_cast<uint8_t*>(workspace) +
                                                   stats_offset(a.r, rows->dtype));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    bool all_done = true;
    rc = done(svl::launch_distill(a, rows->dtype, workspace, &all_done, s));
    if (rc != SV_OK || all_done) return rc;
    return done(svl::launch_distill_grad(a, rows->dtype, true, s));
}

SV_EXPORT int sv_distill_backward(const sv_logit_rows* rows, const int32_t* teacher_tokens,
                                  const float* teacher_logprobs, int64_t k, int tail,
                                  const float* row_stats, const float* grad_loss, void* grad,
                                  int64_t grad_outer_stride, int64_t grad_inner_stride,
                                  void* stream)
{
    svl::DistillArgs a{};
    int rc = check_rows(rows, &a.r);
    if (rc == SV_OK) rc = check_teacher(a.r, teacher_tokens, teacher_logprobs, k, tail);
    if (rc == SV_OK) rc = check_grad(rows, grad, grad_outer_stride, grad_inner_stride, &a.grad);
    if (rc != SV_OK) return rc;
    if (a.r.rows > 0 && (row_stats == nullptr || grad_loss == nullptr)) return SV_ERR_ARG;
    if (!aligned(row_stats, 16) || !aligned(grad_loss, 4)) return SV_ERR_ALIGN;
    if (a.r.rows == 0) return SV_OK;
    a.ids = teacher_tokens;
    a.logp = teacher_logprobs;
    a.k = static_cast<int32_t>(k);
    a.bucket = tail == SV_TAIL_BUCKET;
    a.weights = grad_loss;
    a.stats = reinterpret_cast<svl::RowStats*>(const_cast<float*>(row_stats));
    return done(
        svl::launch_distill_grad(a, rows->dtype, false, static_cast<cudaStream_t>(stream)));
}
