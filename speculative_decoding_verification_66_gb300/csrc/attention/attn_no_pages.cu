// attn_no_pages.cu -- attention over a cache without pages: there is nothing to attend
// to, and no tensor map for the other kernels' copies. Rows of every sequence
// become NaN, and the statuses say why. Also the statuses of calls without rows.
#include "attn_internal.h"

namespace sva {
namespace {

constexpr int kThreads = 128;

template <class T>
__global__ void __launch_bounds__(kThreads) no_pages_kernel(const Attn a)
{
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const uint32_t nan2 = narrow2(nan, nan, T());
    for (int64_t b = blockIdx.x; b < a.c.B; b += gridDim.x) {
        const Seq q = own_seq_of(a.c, static_cast<int>(b), a.tokens, a.max_chunk);
        if (a.status != nullptr && threadIdx.x == 0)
            a.status[b] = q.bad ? q.bad : q.count > 0 ? kBadPage : 0;
        const int64_t row0 = static_cast<int64_t>(q.start) * a.Hq;
        const int64_t rows = static_cast<int64_t>(q.count) * a.Hq;
        uint32_t* o = reinterpret_cast<uint32_t*>(a.out) + row0 * a.c.D / 2;
        for (int64_t i = threadIdx.x; i < rows * a.c.D / 2; i += kThreads) o[i] = nan2;
        if (a.lse != nullptr)
            for (int64_t i = threadIdx.x; i < rows; i += kThreads) a.lse[row0 + i] = nan;
    }
}

}  // namespace

cudaError_t launch_attention_no_pages(const Attn& a, bool f16, cudaStream_t s)
{
    const unsigned blocks = static_cast<unsigned>(a.c.B < 1024 ? a.c.B : 1024);
    if (f16)
        no_pages_kernel<F16><<<blocks, kThreads, 0, s>>>(a);
    else
        no_pages_kernel<Bf16><<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace sva
