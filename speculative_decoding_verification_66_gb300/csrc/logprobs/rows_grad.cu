// rows_grad.cu -- gradients of rows of logits from what the forward pass kept of
// them.
//
// Both gradients are e (A + B t) with t = (x - M) c and e = 2^t: for log
// probabilities and entropy p (c - a - b (log p + H)) / T, with p = e / S and
// log p + H = t ln 2 + (H - log S); for distillation B = 0. What differs at single
// tokens (the given one, the teacher's) is written over it afterwards by the block
// that has the token in its piece, a barrier later.
//
// One read and one write of 16-byte vectors and some seven instructions an element:
// bound by memory. A block takes a piece of a row.
#include "lp_finish.cuh"

namespace svl {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kUnroll = 4;      // vectors that a thread has in flight

// This block's piece of a row.
struct Piece {
    int32_t row;
    int32_t first, end;      // vectors of the gradient's row
};

struct GradPlan {
    int32_t pieces;          // of a row
    int32_t piece;           // vectors
};

// The logits under vector j of the gradient.
template <int DT>
__device__ __forceinline__ uint4 ld_under(const Vecs& in, const Vecs& out, Shift sh, int32_t j,
                                          int32_t V)
{
    if (sh.shift == 0) return ld_vec<DT>(in, j, V);
    const int32_t i = j + sh.step;
    // (vectors around the row's: -inf, nothing is loaded)
    const uint4 a = i < 0 ? ld_vec<DT>(in, in.n, V) : ld_vec<DT>(in, i, V);
    const uint4 b = ld_vec<DT>(in, i + 1, V);
    return shifted(a, b, sh.shift * kElem<DT>);
}

// e (A + B t) over a piece.
template <int DT, bool LINEAR>
__device__ __forceinline__ void grad_piece(const Vecs& in, const Vecs& out, int32_t first,
                                           int32_t end, int32_t V, float M, float c, float A,
                                           float B)
{
    constexpr int P = kPerVec<DT> / 2;
    const Shift sh = shift_of<DT>(in, out);
    const uint64_t m2 = pack2(-M, -M), c2 = pack2(c, c), A2 = pack2(A, A), B2 = pack2(B, B);
    for (int32_t j0 = first + threadIdx.x; j0 < end; j0 += kUnroll * blockDim.x) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t j = j0 + u * blockDim.x;
            if (j < end) v[u] = ld_under<DT>(in, out, sh, j, V);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t j = j0 + u * blockDim.x;
            if (j >= end) break;
            uint64_t p[P];
            widen<DT>(v[u], p);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float t0, t1;
                unpack2(mul2(add2(p[i], m2), c2), t0, t1);
                if (LINEAR) {
                    // (masked logits: 0 times a number and not times -inf)
                    t0 = fmaxf(t0, -1000.f);
                    t1 = fmaxf(t1, -1000.f);
                }
                const uint64_t e = pack2(ex2(t0), ex2(t1));
                p[i] = mul2(e, LINEAR ? fma2(B2, pack2(t0, t1), A2) : A2);
            }
            st_vec<DT>(out, j, V, narrow<DT>(p));
        }
    }
}

__device__ __forceinline__ Piece my_piece(const GradPlan& g, int32_t n)
{
    Piece p;
    p.row = blockIdx.x / g.pieces;
    const int64_t first = static_cast<int64_t>(blockIdx.x - p.row * g.pieces) * g.piece;
    p.first = static_cast<int32_t>(min(first, static_cast<int64_t>(n)));
    p.end = static_cast<int32_t>(min(first + g.piece, static_cast<int64_t>(n)));
    return p;
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads)
    logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a, const GradPlan plan)
{
    const int32_t row = blockIdx.x / plan.pieces, V = a.r.V;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const Vecs out = vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V);
    const Piece pc = my_piece(plan, out.n);
    const RowStats st = a.stats[row];
    if (st.kind != kRowGood) {
        fill<DT>(out, pc.first, pc.end, V, st.kind == kRowBad ? nan() : 0.f);
        return;
    }
    const float da = a.a == nullptr ? 0.f : a.a[row];
    const float db = a.b == nullptr ? 0.f : a.b[row];
    const float dc = a.c == nullptr ? 0.f : a.c[row];
    const float s = st.scale * a.r.inv_t;
    const float A = (dc - da - db * st.mean) * s, B = -db * kLn2 * s;
    // The token's own gradient, where it is in this piece: its logit is read before anything
    // is written, over the logits perhaps.
    const int32_t token = a.tokens == nullptr ? -1 : a.tokens[row];
    const int64_t at = token < 0 ? -1 : (static_cast<int64_t>(token) + out.head) / kPerVec<DT>;
    const bool mine = at >= pc.first && at < pc.end;
    float own = 0.f;
    if (mine) {
        const uint8_t* x = in.a0 + in.head * kElem<DT>;
        const float t = fmaxf((load_one<DT>(x, token) - st.M) * a.r.c, -1000.f);
        own = fmaf(da, a.r.inv_t, ex2(t) * fmaf(B, t, A));
        __syncthreads();
    }
    if (db == 0.f)
        grad_piece<DT, false>(in, out, pc.first, pc.end, V, st.M, a.r.c, A, 0.f);
    else
        grad_piece<DT, true>(in, out, pc.first, pc.end, V, st.M, a.r.c, A, B);
    if (mine) {
        __syncthreads();
        if (threadIdx.x == 0) store_one<DT>(out.a0 + out.head * kElem<DT>, token, own);
    }
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads)
    distill_grad_kernel(const __grid_constant__ DistillArgs a, const GradPlan plan)
{
    __shared__ int32_t id[SV_MAX_TOP];
    __shared__ float logp[SV_MAX_TOP];
    __shared__ float own[SV_MAX_TOP];
    const int32_t row = blockIdx.x / plan.pieces, V = a.r.V;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const Vecs out = vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V);
    const Piece pc = my_piece(plan, out.n);
    const RowStats st = a.stats[row];
    if (st.kind != kRowGood) {
        fill<DT>(out, pc.first, pc.end, V, st.kind == kRowBad ? nan() : 0.f);
        return;
    }
    const float w = a.weights[row] * a.r.inv_t;
    // Entries in this piece. (The row is good: its tokens are in range.)
    int some = 0;
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        const int64_t at = static_cast<int64_t>(row) * a.k + j;
        int32_t v = a.ids[at];
        logp[j] = a.logp[at];
        const int64_t vec = (static_cast<int64_t>(v) + out.head) / kPerVec<DT>;
        if (v < 0 || v >= V || vec < pc.first || vec >= pc.end) v = -1;
        id[j] = v;
        some |= v >= 0;
    }
    some = __syncthreads_or(some);
    if (some) {
        const uint8_t* x = in.a0 + in.head * kElem<DT>;
        for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
            const int32_t v = id[j];
            if (v < 0) continue;
            float p = 0.f;  // (entries of one token: each finds the same sum)
            for (int i = 0; i < a.k; ++i)
                if (id[i] == v) p += expf(logp[i] - st.shift);
            const float e = ex2((load_one<DT>(x, v) - st.listed_M) * a.r.c);
            own[j] = w * (st.listed * e - p * st.inv);
        }
        __syncthreads();
    }
    grad_piece<DT, false>(in, out, pc.first, pc.end, V, st.M, a.r.c, w * st.scale, 0.f);
    if (some) {
        __syncthreads();
        for (int j = threadIdx.x; j < a.k; j += blockDim.x)
            if (id[j] >= 0) store_one<DT>(out.a0 + out.head * kElem<DT>, id[j], own[j]);
    }
}

// A thread moves up to eight vectors, in blocks of 32 to 256 threads: short rows leave few
// threads idle, long ones are cut where a block's start no longer shows.
template <typename Kernel, typename Args>
cudaError_t launch(Kernel k, const Args& a, int per_vec, cudaStream_t s)
{
    const int64_t n = (a.r.V + per_vec - 1) / per_vec + 1;
    int threads = 32;
    while (threads < kMaxThreads && threads * kUnroll < n) threads *= 2;
    GradPlan g;
    g.piece = threads * 2 * kUnroll;
    int64_t pieces = (n + g.piece - 1) / g.piece;
    while (pieces * a.r.rows >= (int64_t(1) << 31)) {
        g.piece *= 2;
        pieces = (n + g.piece - 1) / g.piece;
    }
    g.pieces = static_cast<int32_t>(pieces);
    k<<<static_cast<unsigned>(pieces * a.r.rows), threads, 0, s>>>(a, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, int dtype, cudaStream_t s)
{
    if (dtype == SV_F32) return launch(logprobs_grad_kernel<SV_F32>, a, 4, s);
    if (dtype == SV_BF16) return launch(logprobs_grad_kernel<SV_BF16>, a, 8, s);
    return launch(logprobs_grad_kernel<SV_F16>, a, 8, s);
}

cudaError_t launch_distill_grad(const DistillArgs& a, int dtype, cudaStream_t s)
{
    if (dtype == SV_F32) return launch(distill_grad_kernel<SV_F32>, a, 4, s);
    if (dtype == SV_BF16) return launch(distill_grad_kernel<SV_BF16>, a, 8, s);
    return launch(distill_grad_kernel<SV_F16>, a, 8, s);
}

}  // namespace svl
