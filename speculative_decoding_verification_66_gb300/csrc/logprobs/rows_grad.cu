// rows_grad.cu -- gradients of rows of logits from what the forward pass kept of
// them: a block a row, element by element.
#include "lp_finish.cuh"

namespace svl {
namespace {

constexpr int kThreads = 256;

template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(const LogprobGradArgs a)
{
    const int32_t row = blockIdx.x;
    const uint8_t* x = row_begin(a.r.x, a.r.inner, row);
    uint8_t* g = row_begin(a.grad, a.r.inner, row);
    const float4 st = a.stats[row];
    if (st.w != kRowGood) {
        const float fill = st.w == kRowBad ? nan() : 0.f;
        for (int64_t v = threadIdx.x; v < a.r.V; v += kThreads) store_one<DT>(g, v, fill);
        return;
    }
    const float da = a.a == nullptr ? 0.f : a.a[row];
    const float db = a.b == nullptr ? 0.f : a.b[row];
    const float dc = a.c == nullptr ? 0.f : a.c[row];
    const int32_t token = a.tokens == nullptr ? -1 : a.tokens[row];
    // p (c - a - b (log p + H)) with p = e / S, log p + H = t ln 2 + (H - log S)
    const float A = (dc - da - db * st.z) * st.y * a.r.inv_t;
    const float B = -db * kLn2 * st.y * a.r.inv_t;
    for (int64_t v = threadIdx.x; v < a.r.V; v += kThreads) {
        const float t = fmaxf((load_one<DT>(x, v) - st.x) * a.r.c, -1000.f);
        float d = ex2(t) * fmaf(B, t, A);
        if (v == token) d = fmaf(da, a.r.inv_t, d);
        store_one<DT>(g, v, d);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const DistillArgs a)
{
    __shared__ Teacher t;
    const int32_t row = blockIdx.x;
    const uint8_t* x = row_begin(a.r.x, a.r.inner, row);
    uint8_t* g = row_begin(a.grad, a.r.inner, row);
    const float4 st = a.stats[row];
    if (st.w != kRowGood) {
        const float fill = st.w == kRowBad ? nan() : 0.f;
        for (int64_t v = threadIdx.x; v < a.r.V; v += kThreads) store_one<DT>(g, v, fill);
        return;
    }
    load_teacher(t, a, row);
    const float w = a.weights[row] * a.r.inv_t;
    const float p_scale = a.bucket ? 1.f : static_cast<float>(1.0 / t.mass);
    const int j = threadIdx.x;
    if (j < SV_MAX_TOP) t.x[j] = t.id[j] >= 0 ? load_one<DT>(x, t.id[j]) : 0.f;
    __syncthreads();
    for (int64_t v = threadIdx.x; v < a.r.V; v += kThreads)
        store_one<DT>(g, v, w * st.z * ex2((load_one<DT>(x, v) - st.x) * a.r.c));
    __syncthreads();
    if (j < SV_MAX_TOP && t.id[j] >= 0)
        store_one<DT>(g, t.id[j],
                      w * (st.y * ex2((t.x[j] - st.x) * a.r.c) - t.p[j] * p_scale));
}

}  // namespace

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, int dtype, cudaStream_t s)
{
    const auto k = dtype == SV_F32    ? logprobs_grad_kernel<SV_F32>
                   : dtype == SV_BF16 ? logprobs_grad_kernel<SV_BF16>
                                      : logprobs_grad_kernel<SV_F16>;
    k<<<a.r.rows, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_distill_grad(const DistillArgs& a, int dtype, cudaStream_t s)
{
    const auto k = dtype == SV_F32    ? distill_grad_kernel<SV_F32>
                   : dtype == SV_BF16 ? distill_grad_kernel<SV_BF16>
                                      : distill_grad_kernel<SV_F16>;
    k<<<a.r.rows, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace svl
