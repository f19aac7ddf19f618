// distill.cu -- divergence of a teacher's entries from rows of logits, and its
// gradient, in one read of the row and one write.
//
// The gradient of an element needs the sum over its whole row, and a row does not fit
// into the registers or the shared memory that a block can have beside others. A cluster
// of up to eight blocks takes the row: each keeps its share in shared memory, the shares'
// maxima and sums and the entries' logits are told to every block of the cluster through
// distributed shared memory, and every block computes the row's few logarithms for itself
// (one barrier over the cluster, where one block's answer to the others would take two).
//
// A thread copies its vectors into shared memory (cp.async) and is the one that reads them
// again, so the copies need no barrier; what does is that the entries' logits are taken out
// of the share, and -inf put in their place: the sums are then over the other tokens, with
// nothing to subtract, and the gradient's loop has no cases. The entries' gradients are
// written over it at the end.
//
// Shares larger than shared memory go through it chunk by chunk, twice; the last chunk of
// the first pass is the first of the second.
#include "lp_finish.cuh"

namespace svl {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxCluster = 8;

struct DistillPlan {
    int32_t cluster;     // blocks of a row
    int32_t share;       // vectors of a block
    int32_t chunk;       // vectors that it holds at a time
};

__device__ __forceinline__ void copy_in(uint8_t* to, const uint8_t* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sv::smem_addr(to)), "l"(from)
                 : "memory");
}

__device__ __forceinline__ void st_shared(uint8_t* p, uint4 v)
{
    *reinterpret_cast<uint4*>(p) = v;
}

// Vectors [first, first + n) of a row to shared memory; waited for by wait_copies, each
// thread for its own.
template <int DT>
__device__ __forceinline__ void load_chunk(uint8_t* room, const Vecs& in, int32_t first, int32_t n,
                                           int32_t V)
{
    for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
        const int32_t at = first + i;
        if (at >= in.full && at < in.full_end)
            copy_in(room + 16 * i, in.a0 + static_cast<int64_t>(at) * 16);
        else
            st_shared(room + 16 * i, ld_edge<DT>(in.a0, at, in.head, V));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Takes the entries' logits out of a chunk (element `first_of` its first vector on).
template <int DT>
__device__ __forceinline__ void take_entries(uint8_t* room, Teacher& t, int32_t k, int64_t begin,
                                             int32_t n, uint32_t& mine)
{
    int turn = 0;
    for (int j = threadIdx.x; j < k; j += blockDim.x, ++turn) {
        const int64_t at = t.id[j] - begin;
        if (t.id[j] < 0 || at < 0 || at >= static_cast<int64_t>(n) * kPerVec<DT>) continue;
        const float x = load_one<DT>(room, at);
        if (!(mine >> turn & 1)) t.x[j] = x;
        mine |= 1u << turn;
        store_one<DT>(room, at, -inf());
    }
}

struct Sum {
    float m, s;      // largest logit; sum of 2^((x - m) c)
};

// The smaller maximum's sum is brought to the larger one's. (-inf: nothing yet.)
__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    Sum r;
    r.m = fmax_nan(a.m, b.m);
    r.s = (a.s > 0.f ? a.s * ex2((a.m - r.m) * c) : 0.f) +
          (b.s > 0.f ? b.s * ex2((b.m - r.m) * c) : 0.f);
    return r;
}

// This thread's part of a chunk: its largest logit, then the sum against it.
template <int DT>
__device__ __forceinline__ Sum sum_chunk(const uint8_t* room, int32_t n, float c)
{
    Sum r{-inf(), 0.f};
    uint32_t top = kNegInf<DT>;
    for (int32_t i = threadIdx.x; i < n; i += blockDim.x)
        top = packed_max<DT>(top, vec_max<DT>(*reinterpret_cast<const uint4*>(room + 16 * i)));
    r.m = halves_max<DT>(top);
    if (!(fabsf(r.m) < inf())) return r;  // nothing but -inf; or a bad row, whose sum is not used
    const uint64_t m2 = pack2(-r.m, -r.m), c2 = pack2(c, c);
    uint64_t s0 = pack2(0.f, 0.f), s1 = s0;
    for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
        uint64_t p[kPerVec<DT> / 2];
        widen<DT>(*reinterpret_cast<const uint4*>(room + 16 * i), p);
#pragma unroll
        for (int q = 0; q < kPerVec<DT> / 2; ++q) {
            float a, b;
            unpack2(mul2(add2(p[q], m2), c2), a, b);
            const uint64_t e = pack2(ex2(a), ex2(b));
            if (q & 1)
                s1 = add2(s1, e);
            else
                s0 = add2(s0, e);
        }
    }
    float a, b;
    unpack2(add2(s0, s1), a, b);
    r.s = a + b;
    return r;
}

template <int DT>
__device__ __forceinline__ void grad_chunk(const uint8_t* room, const Vecs& in, const Vecs& out,
                                           int32_t first, int32_t n, int32_t V, float M, float c,
                                           float A)
{
    constexpr int P = kPerVec<DT> / 2;
    const uint64_t m2 = pack2(-M, -M), c2 = pack2(c, c), A2 = pack2(A, A);
    const bool same = in.head == out.head;
    for (int32_t i = threadIdx.x; i < n; i += blockDim.x) {
        uint64_t p[P];
        widen<DT>(*reinterpret_cast<const uint4*>(room + 16 * i), p);
#pragma unroll
        for (int q = 0; q < P; ++q) {
            float a, b;
            unpack2(mul2(add2(p[q], m2), c2), a, b);
            p[q] = mul2(pack2(ex2(a), ex2(b)), A2);
        }
        const int32_t at = first + i;
        if (same) {
            st_vec<DT>(out, at, V, narrow<DT>(p));
        } else {
            // Rows that do not begin equally far from a boundary: element by element.
            uint8_t* g = out.a0 + out.head * kElem<DT>;
            const int64_t v0 = first_of<DT>(in, at);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float a, b;
                unpack2(p[q], a, b);
                const int64_t v = v0 + 2 * q;
                if (v >= 0 && v < V) store_one<DT>(g, v, a);
                if (v + 1 >= 0 && v + 1 < V) store_one<DT>(g, v + 1, b);
            }
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
    distill_kernel(const __grid_constant__ DistillArgs a, const DistillPlan plan)
{
    extern __shared__ __align__(16) uint8_t room[];
    __shared__ Teacher t;
    __shared__ Sum part[kThreads / 32];
    __shared__ float from_m[kMaxCluster], from_s[kMaxCluster];
    const int C = plan.cluster;
    const int32_t row = blockIdx.x / C, rank = blockIdx.x - row * C, V = a.r.V;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float c = a.r.c;
    // (that all blocks of the cluster run is known to each before it writes to another)
    if (C > 1) cluster_arrive();
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const int64_t lo = static_cast<int64_t>(rank) * plan.share;
    const int32_t first = static_cast<int32_t>(min(lo, static_cast<int64_t>(in.n)));
    const int32_t end = static_cast<int32_t>(min(lo + plan.share, static_cast<int64_t>(in.n)));
    const int32_t chunks = (end - first + plan.chunk - 1) / plan.chunk;
    const bool has_grad = a.grad.base != nullptr;
    const Vecs out = has_grad ? vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V) : in;
    int kind = kRowGood;
    uint32_t mine = 0;  // this thread's entries that lie in this block's share
    int32_t held = 0;   // the chunk in shared memory

    if (!read_teacher(t, a, row)) {
        kind = kRowSkipped;
        if (rank == 0 && threadIdx.x == 0) finish_distill_skipped(a, row);
        if (C > 1) cluster_wait();
    } else {
        if (chunks > 0) load_chunk<DT>(room, in, first, min(plan.chunk, end - first), V);
        make_teacher(t, a);
        Sum mine_sum{-inf(), 0.f};
        for (int32_t ch = 0; ch < chunks; ++ch) {
            const int32_t at = first + ch * plan.chunk, n = min(plan.chunk, end - at);
            if (ch > 0) load_chunk<DT>(room, in, at, n, V);
            wait_copies();
            __syncthreads();
            take_entries<DT>(room, t, a.k, first_of<DT>(in, at), n, mine);
            __syncthreads();
            mine_sum = join(mine_sum, sum_chunk<DT>(room, n, c), c);
            held = ch;
            if (ch + 1 < chunks) __syncthreads();
        }
        // The warp's, the block's and the cluster's sums.
        for (int off = 16; off > 0; off >>= 1) {
            Sum o;
            o.m = __shfl_xor_sync(0xFFFFFFFFu, mine_sum.m, off);
            o.s = __shfl_xor_sync(0xFFFFFFFFu, mine_sum.s, off);
            mine_sum = join(mine_sum, o, c);
        }
        if (lane == 0) part[warp] = mine_sum;
        if (C > 1) cluster_wait();
        __syncthreads();
        Sum total = part[0];
        for (int w = 1; w < warps; ++w) total = join(total, part[w], c);
        if (C > 1) {
            if (threadIdx.x < C) {
                st_cluster(&from_m[rank], threadIdx.x, total.m);
                st_cluster(&from_s[rank], threadIdx.x, total.s);
            }
            int turn = 0;
            for (int j = threadIdx.x; j < a.k; j += blockDim.x, ++turn)
                if (mine >> turn & 1)
                    for (int r = 0; r < C; ++r)
                        if (r != rank) st_cluster(&t.x[j], r, t.x[j]);
            cluster_arrive();
            cluster_wait();
            total = {from_m[0], from_s[0]};
            for (int r = 1; r < C; ++r) total = join(total, {from_m[r], from_s[r]}, c);
        }
        kind = finish_distill(t, a, row, total.m, total.s, rank == 0);
    }
    if (!has_grad) return;
    if (kind != kRowGood) {
        const int32_t g0 = static_cast<int32_t>(min(lo, static_cast<int64_t>(out.n)));
        const int32_t g1 = static_cast<int32_t>(min(lo + plan.share, static_cast<int64_t>(out.n)));
        fill<DT>(out, g0, g1, V, kind == kRowBad ? nan() : 0.f);
        return;
    }
    const float w = (a.weights == nullptr ? 1.f : a.weights[row]) * a.r.inv_t;
    for (int32_t ch = chunks - 1; ch >= 0; --ch) {
        const int32_t at = first + ch * plan.chunk, n = min(plan.chunk, end - at);
        if (ch != held) {
            load_chunk<DT>(room, in, at, n, V);
            wait_copies();
        }
        grad_chunk<DT>(room, in, out, at, n, V, t.M, c, w * t.scale);
    }
    __syncthreads();
    int turn = 0;
    for (int j = threadIdx.x; j < a.k; j += blockDim.x, ++turn)
        if (mine >> turn & 1)
            store_one<DT>(out.a0 + out.head * kElem<DT>, t.id[j],
                          w * (t.listed * ex2((t.x[j] - t.listed_M) * c) - t.p[j]));
}

template <int DT>
cudaError_t launch(const DistillArgs& a, cudaStream_t s)
{
    constexpr int64_t kChunk = 4096;      // 64 KB: three blocks an SM
    constexpr int64_t kMaxChunk = 6656;   // 104 KB: two
    constexpr int64_t kBlocks = 304;      // two an SM
    const int64_t n = (a.r.V + kPerVec<DT> - 1) / kPerVec<DT> + 1;
    int64_t C = 1;
    while (C < kMaxCluster && a.r.rows * C * 2 < (int64_t(1) << 31) &&
           ((n + C - 1) / C > kChunk || (a.r.rows * C < kBlocks && n / C > kThreads)))
        C *= 2;
    DistillPlan p;
    p.cluster = static_cast<int32_t>(C);
    p.share = static_cast<int32_t>((n + C - 1) / C);
    p.chunk = static_cast<int32_t>(p.share <= kMaxChunk ? p.share : kChunk);
    int threads = 32;
    while (threads < kThreads && threads * 4 < p.share) threads *= 2;
    auto* k = distill_kernel<DT>;
    if (p.chunk * 16 > 45000) {  // (beside the static part, more than is allowed unasked)
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kMaxChunk * 16));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.r.rows * C));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.chunk) * 16;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(C);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a, p);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t s)
{
    return dtype == SV_F32 ? launch<SV_F32>(a, s) : dtype == SV_BF16 ? launch<SV_BF16>(a, s)
                                                                      : launch<SV_F16>(a, s);
}

}  // namespace svl
