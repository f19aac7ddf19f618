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
// bound by memory. A block takes a piece of a row. 4096 rows of 128256 bfloat16, 2.1 GB: 313 us
// (6.7 TB/s), or 322 with a teacher's 32 entries a row; 1024 rows 86 and 92.
#include "lp_finish.cuh"
#include "lp_stream.cuh"

namespace svl {
namespace {

constexpr int kMaxThreads = kGradWarps * 32;

// This block's turns in its row.
struct Piece {
    int32_t first, end;      // of the block
    int32_t mine, step;      // of the warp
};

// The last row first: the forward pass has read it last, and has left it in L2.
__device__ __forceinline__ int32_t row_of(const GradPlan& g, int32_t rows)
{
    return rows - 1 - static_cast<int32_t>(blockIdx.x / g.pieces);
}

__device__ __forceinline__ Piece my_piece(const GradPlan& g, int32_t vectors)
{
    Piece p;
    const int32_t tiles = tiles_of(vectors);
    const int64_t first = static_cast<int64_t>(blockIdx.x % g.pieces) * g.piece;
    p.first = static_cast<int32_t>(min(first, static_cast<int64_t>(tiles)));
    p.end = static_cast<int32_t>(min(first + g.piece, static_cast<int64_t>(tiles)));
    p.mine = p.first + (threadIdx.x >> 5);
    p.step = blockDim.x >> 5;
    return p;
}

// (not through the read-only path: another kernel may still have been writing when this one began)
__device__ __forceinline__ RowStats load_stats(const RowStats* p)
{
    const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads)
    logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a, const GradPlan plan)
{
    const int32_t row = row_of(plan, a.r.rows), V = a.r.V;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const Vecs out = vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V);
    const Piece pc = my_piece(plan, out.n);
    const RowStats st = a.stats[row];
    // The kind is of the forward call's tokens, and these may be others.
    const int32_t token = a.tokens == nullptr ? 0 : a.tokens[row];
    const bool out_of_range = token < -1 || token >= V;
    if (st.kind != kRowGood || token == -1 || out_of_range) {
        const bool bad = st.kind == kRowBad || out_of_range;
        fill_tiles<DT>(out, pc.mine, pc.step, pc.end, V, bad ? nan() : 0.f);
        return;
    }
    const float da = a.a == nullptr ? 0.f : a.a[row];
    const float db = a.b == nullptr ? 0.f : a.b[row];
    const float dc = a.c == nullptr ? 0.f : a.c[row];
    const float s = st.scale * a.r.inv_t;
    const float A = (dc - da - db * st.mean) * s, B = -db * kLn2 * s;
    // The token's own gradient, where it is in this piece: its logit is read before anything
    // is written, over the logits perhaps.
    const int64_t at =
        a.tokens == nullptr ? -1 : (static_cast<int64_t>(token) + out.head) / (kPerVec<DT> * kTile);
    const bool mine = at >= pc.first && at < pc.end;
    float own = 0.f;
    if (mine) {
        const uint8_t* x = in.a0 + in.head * kElem<DT>;
        const float t = fmaxf((load_one<DT>(x, token) - st.M) * a.r.c, -1000.f);
        own = fmaf(da, a.r.inv_t, ex2(t) * fmaf(B, t, A));
        __syncthreads();
    }
    if (db == 0.f)
        grad_tiles<DT, false>(in, out, pc.mine, pc.step, pc.end, V, st.M, a.r.c, A, 0.f);
    else
        grad_tiles<DT, true>(in, out, pc.mine, pc.step, pc.end, V, st.M, a.r.c, A, B);
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
    const int32_t row = row_of(plan, a.r.rows), V = a.r.V;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const Vecs out = vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V);
    const Piece pc = my_piece(plan, out.n);
    sv::pdl_wait();   // (behind sv_distill's sums this kernel is launched before they end)
    const RowStats st = load_stats(a.stats + row);
    if (st.kind != kRowGood) {
        fill_tiles<DT>(out, pc.mine, pc.step, pc.end, V, st.kind == kRowBad ? nan() : 0.f);
        return;
    }
    const float w = (a.weights == nullptr ? 1.f : a.weights[row]) * a.r.inv_t;
    // Entries in this piece. (The row is good: its tokens are in range.)
    int some = 0;
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        const int64_t at = static_cast<int64_t>(row) * a.k + j;
        int32_t v = a.ids[at];
        logp[j] = a.logp[at];
        const int64_t tile = (static_cast<int64_t>(v) + out.head) / (kPerVec<DT> * kTile);
        if (v < 0 || v >= V || tile < pc.first || tile >= pc.end) v = -1;
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
    grad_tiles<DT, false>(in, out, pc.mine, pc.step, pc.end, V, st.M, a.r.c, w * st.scale, 0.f);
    if (some) {
        __syncthreads();
        for (int j = threadIdx.x; j < a.k; j += blockDim.x)
            if (id[j] >= 0) store_one<DT>(out.a0 + out.head * kElem<DT>, id[j], own[j]);
    }
}

template <typename Kernel, typename Args>
cudaError_t launch(Kernel k, const Args& a, int per_vec, cudaStream_t s, bool early = false)
{
    int warps;
    const GradPlan g = grad_plan_of(a.r.rows, most_tiles(a.r.V, per_vec), &warps);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(g.pieces) * static_cast<unsigned>(a.r.rows));
    cfg.blockDim = dim3(warps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a, g);
}

}  // namespace

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, int dtype, cudaStream_t s)
{
    if (dtype == SV_F32) return launch(logprobs_grad_kernel<SV_F32>, a, 4, s);
    if (dtype == SV_BF16) return launch(logprobs_grad_kernel<SV_BF16>, a, 8, s);
    return launch(logprobs_grad_kernel<SV_F16>, a, 8, s);
}

cudaError_t launch_distill_grad(const DistillArgs& a, int dtype, bool behind, cudaStream_t s)
{
    if (dtype == SV_F32) return launch(distill_grad_kernel<SV_F32>, a, 4, s, behind);
    if (dtype == SV_BF16) return launch(distill_grad_kernel<SV_BF16>, a, 8, s, behind);
    return launch(distill_grad_kernel<SV_F16>, a, 8, s, behind);
}

}  // namespace svl
