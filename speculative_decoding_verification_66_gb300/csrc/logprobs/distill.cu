// distill.cu -- divergence of a teacher's entries from rows of logits, and its
// gradient: a block a row, element by element.
#include "lp_finish.cuh"

namespace svl {
namespace {

constexpr int kThreads = 256;

template <typename F>
__device__ __forceinline__ float block_reduce(float x, float* shared, F f)
{
    for (int off = 16; off > 0; off >>= 1) x = f(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    x = shared[0];
    for (int w = 1; w < kThreads / 32; ++w) x = f(x, shared[w]);
    return x;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a)
{
    __shared__ Teacher t;
    __shared__ float part[kThreads / 32];
    const int32_t row = blockIdx.x;
    const int tid = threadIdx.x, V = a.r.V;
    const uint8_t* x = row_begin(a.r.x, a.r.inner, row);
    uint8_t* g = a.grad.base == nullptr ? nullptr : row_begin(a.grad, a.r.inner, row);
    load_teacher(t, a, row);
    int kind = t.status != 0 ? kRowBad : t.distinct == 0 ? kRowSkipped : kRowGood;
    int status = t.status;
    float M = -inf();
    if (kind != kRowSkipped) {
        for (int64_t v = tid; v < V; v += kThreads) M = fmax_nan(M, load_one<DT>(x, v));
        M = block_reduce(M, part, [](float p, float q) { return fmax_nan(p, q); });
        if (!(fabsf(M) < inf())) {
            kind = kRowBad;
            status |= SV_SEQ_NONFINITE;
        }
    }
    if (kind != kRowGood) {
        if (tid == 0) finish_distill_plain(a, row, kind, status);
        if (g != nullptr)
            for (int64_t v = tid; v < V; v += kThreads)
                store_one<DT>(g, v, kind == kRowBad ? nan() : 0.f);
        return;
    }
    float S = 0.f;
    for (int64_t v = tid; v < V; v += kThreads) {
        bool listed = false;
        for (int i = 0; i < a.k; ++i) listed |= t.id[i] == v;
        if (!listed) S += ex2((load_one<DT>(x, v) - M) * a.r.c);
    }
    S = block_reduce(S, part, [](float p, float q) { return p + q; });
    if (tid < SV_MAX_TOP) t.x[tid] = t.id[tid] >= 0 ? load_one<DT>(x, t.id[tid]) : 0.f;
    __syncthreads();
    finish_distill(t, a, row, M, S);
    if (g == nullptr) return;
    const float w = (a.weights == nullptr ? 1.f : a.weights[row]) * a.r.inv_t;
    for (int64_t v = tid; v < V; v += kThreads)
        store_one<DT>(g, v, w * t.others * ex2((load_one<DT>(x, v) - M) * a.r.c));
    __syncthreads();
    if (tid < SV_MAX_TOP && t.id[tid] >= 0)
        store_one<DT>(g, t.id[tid], w * (t.listed * ex2((t.x[tid] - M) * a.r.c) - t.p[tid]));
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t s)
{
    const auto k = dtype == SV_F32    ? distill_kernel<SV_F32>
                   : dtype == SV_BF16 ? distill_kernel<SV_BF16>
                                      : distill_kernel<SV_F16>;
    k<<<a.r.rows, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace svl
