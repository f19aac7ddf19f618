// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives:
// a block a row, element by element, in as many passes as it takes.
#include "lp_finish.cuh"

namespace svl {
namespace {

constexpr int kThreads = 256;

// Sum or maximum over a block; all threads get it.
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
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a)
{
    __shared__ float part[kThreads / 32];
    __shared__ unsigned long long best;
    const int32_t row = blockIdx.x;
    const int tid = threadIdx.x, V = a.r.V;
    const auto add = [](float x, float y) { return x + y; };
    const auto most = [](float x, float y) { return fmax_nan(x, y); };
    const int32_t token = a.tokens == nullptr ? 0 : a.tokens[row];
    const uint8_t* x = row_begin(a.r.x, a.r.inner, row);
    int kind = token == -1 ? kRowSkipped : token < 0 || token >= V ? kRowBad : kRowGood;
    int status = kind == kRowBad ? SV_SEQ_BAD_TOKEN : 0;
    float M = -inf();
    if (kind != kRowSkipped) {
        for (int64_t v = tid; v < V; v += kThreads) M = fmax_nan(M, load_one<DT>(x, v));
        M = block_reduce(M, part, most);
        if (!(fabsf(M) < inf())) {
            kind = kRowBad;
            status |= SV_SEQ_NONFINITE;
        }
    }
    if (kind != kRowGood) {
        if (tid == 0) finish_plain(a, row, kind, status);
        finish_plain_top(a, row, kind, tid, kThreads);
        return;
    }
    const float x_t = load_one<DT>(x, token);
    float S = 0.f, E = 0.f, ahead = 0.f;
    for (int64_t v = tid; v < V; v += kThreads) {
        const float y = load_one<DT>(x, v);
        const float t = fmaxf((y - M) * a.r.c, -1000.f);
        const float e = ex2(t);
        S += e;
        E += e * t;
        ahead += y > x_t || (y == x_t && v < token) ? 1.f : 0.f;
    }
    S = block_reduce(S, part, add);
    E = block_reduce(E, part, add);
    ahead = block_reduce(ahead, part, add);
    const double log_s = log_wide(S);
    if (tid == 0) finish_row(a, row, M, S, E, x_t, static_cast<int>(ahead), log_s);
    // Place by place: the largest below the last one taken.
    unsigned long long last = ~0ull;
    for (int j = 0; j < a.k; ++j) {
        if (tid == 0) best = 0;
        __syncthreads();
        unsigned long long mine = 0;
        for (int v = tid; v < V; v += kThreads) {
            const unsigned long long key =
                (static_cast<unsigned long long>(ordered(load_one<DT>(x, v))) << 32) |
                (0xFFFFFFFFu - static_cast<uint32_t>(v));
            if (key < last && key > mine) mine = key;
        }
        atomicMax(&best, mine);
        __syncthreads();
        last = best;
        if (tid == 0) {
            const int64_t at = static_cast<int64_t>(row) * a.k + j;
            const float y = unordered(static_cast<uint32_t>(last >> 32));
            a.top_tokens[at] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(last));
            a.top_logprobs[at] = static_cast<float>(log_prob(y, M, a.r.c, log_s));
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s)
{
    const auto k = dtype == SV_F32    ? logprobs_kernel<SV_F32>
                   : dtype == SV_BF16 ? logprobs_kernel<SV_BF16>
                                      : logprobs_kernel<SV_F16>;
    k<<<a.r.rows, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace svl
