// attn_rows.cu -- attention of the new tokens, one warp a query row, one key at a
// time. For caches that the tensor copies of the other kernels cannot describe: no
// pages at all, or strides that a tensor map does not take. A row's keys come one
// behind the other, so it is bound by the latency of its loads: 64 x 5 tokens take
// 3.2 ms where attn_tiles.cu takes 0.13.
#include "attn_internal.h"

namespace sva {
namespace {

constexpr int kWarps = 4;

template <class T, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const Attn a)
{
    const Cache& c = a.c;
    const int lane = threadIdx.x & 31;
    if (a.status != nullptr)
        for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < c.B;
             b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
            const int bad = seq_of(c, static_cast<int>(b), a.tokens, a.max_chunk).bad;
            if (bad) atomicOr(a.status + b, bad);
        }
    const int64_t r = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5);
    const int64_t t = r / a.Hq;
    const int h = static_cast<int>(r - t * a.Hq);
    if (t >= a.tokens) return;
    const int b = find_seq(c.starts, c.B, t, lane);
    const Seq q = seq_of(c, b, a.tokens, a.max_chunk);
    if (t < q.start || t - q.start >= q.count) return;
    float m = 0.f, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool ok = !q.bad;
    if (ok) {
        const int64_t pos = q.cached + (t - q.start);
        ok = attend_row<T, E4M3>(a, b, h / a.G, a.q + t * a.q_token + h * a.q_head,
                                 first_key(a, pos), pos + 1, lane, &m, &l, o);
        if (!ok && a.status != nullptr && lane == 0) atomicOr(a.status + b, kBadPage);
    }
    const float inv = ok ? 1.f / l : __uint_as_float(0x7FFFFFFFu);
    if (lane * 8 < c.D)
        *reinterpret_cast<uint4*>(a.out + (r * c.D + lane * 8) * 2) =
            make_uint4(narrow2(o[0] * inv, o[1] * inv, T()), narrow2(o[2] * inv, o[3] * inv, T()),
                       narrow2(o[4] * inv, o[5] * inv, T()), narrow2(o[6] * inv, o[7] * inv, T()));
    if (a.lse != nullptr && lane == 0)
        a.lse[r] = ok ? fmaf(m, kLn2, logf(l)) : __uint_as_float(0x7FFFFFFFu);
}

template <class T, bool E4M3>
cudaError_t launch(const Attn& a, cudaStream_t s)
{
    const int64_t blocks = (a.tokens * a.Hq + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    rows_kernel<T, E4M3><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_rows(const Attn& a, bool f16, bool e4m3, cudaStream_t s)
{
    if (f16) return e4m3 ? launch<F16, true>(a, s) : launch<F16, false>(a, s);
    return e4m3 ? launch<Bf16, true>(a, s) : launch<Bf16, false>(a, s);
}

}  // namespace sva
