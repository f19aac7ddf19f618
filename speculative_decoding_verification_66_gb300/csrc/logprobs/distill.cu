// distill.cu -- divergence of a teacher's entries from rows of logits, and its
// gradient, in one read of memory and one write.
//
// The gradient of an element needs the sum over its whole row first. A block goes through
// its row twice, and the second time finds it in L2: what the resident blocks have of rows
// is kept below the cache's size. (Rows held in a cluster's shared memory, 64 KB a block,
// read L2 once less and took more than twice as long: what a row waits for -- its teacher,
// barriers, a few logarithms -- has little to hide behind where a row fills an SM.)
//
// With SV_TAIL_BUCKET the sum over the tokens without entries must not be a difference:
// where a teacher's few tokens have nearly all of the student's probability too, nothing
// would be left of it. A bitmap of the entries' tokens in shared memory has a byte for each
// vector of eight; a warp looks at its vectors' bytes and takes out what is marked, which is
// rare. (Renormalised or not: the sum is over the others, and the entries are added.)
//
// The entries' gradients are written over what the loop wrote for them, a barrier later.
//
// A row is taken by a block, or by a cluster of up to eight where there are few rows or they
// are long: each block tells all others its part's maximum and sum, and all find the row's
// few logarithms for themselves (one barrier over the cluster; an answer would take two).
#include "lp_finish.cuh"
#include "lp_stream.cuh"

namespace svl {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 8;
// A bitmap's words, and the elements that they are for: longer rows take turns with it.
constexpr int32_t kMapWords = 8192;

struct DistillPlan {
    int32_t cluster;     // blocks of a row
    int32_t words;       // of the bitmap
};

// Sets or clears the marks of the entries from position `begin` on.
template <bool SET>
__device__ __forceinline__ void mark(uint32_t* map, const Teacher& t, int32_t k, int32_t head,
                                     int64_t begin, int32_t words)
{
    for (int j = threadIdx.x; j < k; j += blockDim.x) {
        const int64_t at = static_cast<int64_t>(t.id[j]) + head - begin;
        if (t.id[j] < 0 || at < 0 || at >= static_cast<int64_t>(words) * 32) continue;
        if (SET)
            atomicOr(&map[at >> 5], 1u << (at & 31));
        else
            map[at >> 5] = 0u;
    }
}

// -inf for the marked elements of a vector.
template <int DT>
__device__ __noinline__ uint4 without(uint4 v, uint32_t marks)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == SV_F32) {
            if (marks >> i & 1) w[i] = kNegInf<DT>;
        } else {
            if (marks >> (2 * i) & 1) w[i] = (w[i] & 0xFFFF0000u) | (kNegInf<DT> & 0xFFFFu);
            if (marks >> (2 * i + 1) & 1) w[i] = (w[i] & 0xFFFFu) | (kNegInf<DT> & 0xFFFF0000u);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The marks of vector i (counted from the bitmap's begin).
template <int DT>
__device__ __forceinline__ uint32_t marks_of(const uint32_t* map, int32_t i)
{
    const uint8_t* b = reinterpret_cast<const uint8_t*>(map);
    return DT == SV_F32 ? b[i >> 1] >> ((i & 1) * 4) & 15u : b[i];
}

template <int DT>
__global__ void __launch_bounds__(kMaxThreads)
    distill_kernel(const __grid_constant__ DistillArgs a, const DistillPlan plan)
{
    extern __shared__ __align__(16) uint32_t map[];
    __shared__ Teacher t;
    __shared__ float part_m[kMaxThreads / 32], part_s[kMaxThreads / 32];
    __shared__ float from_m[kMaxCluster], from_s[kMaxCluster];
    const int C = plan.cluster;
    const int32_t row = blockIdx.x / C, rank = blockIdx.x - row * C, V = a.r.V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float c = a.r.c;
    const int32_t first_tile = rank * warps + warp, step_tiles = C * warps;
    // (that all blocks of the cluster run is known to each before it writes to another)
    if (C > 1) cluster_arrive();
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const bool has_grad = a.grad.base != nullptr;
    const Vecs out = has_grad ? vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V) : in;
    for (int i = threadIdx.x; i < plan.words; i += blockDim.x) map[i] = 0u;
    int kind = kRowSkipped;
    if (!read_teacher(t, a, row)) {
        if (rank == 0 && threadIdx.x == 0) finish_distill_skipped(a, row);
        if (C > 1) cluster_wait();
    } else {
        make_teacher(t, a);
        const uint8_t* x = in.a0 + in.head * kElem<DT>;
        for (int j = threadIdx.x; j < a.k; j += blockDim.x)
            if (t.id[j] >= 0) t.x[j] = load_one<DT>(x, t.id[j]);
        Running st;
        start(st);
        const float step = 16.f / c, low = lowest_of<DT>(c);
        const int32_t tiles = tiles_of(in.n);
        const int32_t span = plan.words * 32 / (kPerVec<DT> * kTile);  // turns of one bitmap
        for (int32_t t0 = 0; t0 < tiles; t0 += span) {
            const int64_t begin = static_cast<int64_t>(t0) * kTile * kPerVec<DT>;
            if (t0 > 0) {
                __syncthreads();
                mark<false>(map, t, a.k, in.head, begin - static_cast<int64_t>(plan.words) * 32,
                            plan.words);
                __syncthreads();
            }
            mark<true>(map, t, a.k, in.head, begin, plan.words);
            __syncthreads();
            int32_t tile = t0 + (first_tile - t0 % step_tiles + step_tiles) % step_tiles;
            for (; tile < min(t0 + span, tiles); tile += step_tiles) {
                const int32_t base = tile * kTile;
                uint4 v[kInFlight];
                ld_tile<DT>(v, in, base, lane, V);
                uint32_t marks[kInFlight];
#pragma unroll
                for (int u = 0; u < kInFlight; ++u)
                    marks[u] = marks_of<DT>(map, base - t0 * kTile + lane + u * 32);
                if ((marks[0] | marks[1] | marks[2] | marks[3]) != 0) {
#pragma unroll
                    for (int u = 0; u < kInFlight; ++u)
                        if (marks[u] != 0) v[u] = without<DT>(v[u], marks[u]);
                }
                uint32_t top = vec_max<DT>(v[0]);
#pragma unroll
                for (int u = 1; u < kInFlight; ++u) top = packed_max<DT>(top, vec_max<DT>(v[u]));
                take<DT, false>(st, v, halves_max<DT>(top), c, step, low);
            }
        }
        const RowSum mine = warp_join(st, 0, c);
        if (lane == 0) {
            part_m[warp] = mine.m;
            part_s[warp] = mine.s;
        }
        if (C > 1) cluster_wait();
        __syncthreads();
        RowSum all{part_m[0], part_s[0], 0.f, 0};
        for (int w = 1; w < warps; ++w) all = join(all, {part_m[w], part_s[w], 0.f, 0}, c);
        if (C > 1) {
            if (threadIdx.x < C) {
                st_cluster(&from_m[rank], threadIdx.x, all.m);
                st_cluster(&from_s[rank], threadIdx.x, all.s);
            }
            cluster_arrive();
            cluster_wait();
            all = {from_m[0], from_s[0], 0.f, 0};
            for (int r = 1; r < C; ++r) all = join(all, {from_m[r], from_s[r], 0.f, 0}, c);
        }
        kind = finish_distill(t, a, row, all.m, all.s, rank == 0);
    }
    if (!has_grad) return;
    const int32_t out_tiles = tiles_of(out.n);
    if (kind != kRowGood) {
        fill_tiles<DT>(out, first_tile, step_tiles, out_tiles, V, kind == kRowBad ? nan() : 0.f);
        return;
    }
    const float w = (a.weights == nullptr ? 1.f : a.weights[row]) * a.r.inv_t;
    grad_tiles<DT, false>(in, out, first_tile, step_tiles, out_tiles, V, t.M, c, w * t.scale, 0.f);
    __syncthreads();
    // The entries in this block's turns.
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        if (t.id[j] < 0) continue;
        const int64_t tile = (static_cast<int64_t>(t.id[j]) + out.head) / (kPerVec<DT> * kTile);
        if (tile / warps % C != rank) continue;
        store_one<DT>(out.a0 + out.head * kElem<DT>, t.id[j],
                      w * (t.listed * ex2((t.x[j] - t.listed_M) * c) - t.p[j]));
    }
}

template <int DT>
cudaError_t launch(const DistillArgs& a, cudaStream_t s)
{
    constexpr int64_t kBlocks = 304;               // two an SM
    constexpr int64_t kPart = int64_t(280) << 10;  // a block's share: twice 152 of it fit in L2
    const int64_t n = (a.r.V + kPerVec<DT> - 1) / kPerVec<DT> + 1;
    const int64_t tiles = tiles_of(n);
    int warps = 1;
    while (warps * 32 < kMaxThreads && warps < tiles) warps *= 2;
    int64_t C = 1;
    while (C < kMaxCluster && a.r.rows * C * 2 < (int64_t(1) << 31) &&
           (n * 16 / C > kPart || (a.r.rows * C < kBlocks && tiles > C * warps)))
        C *= 2;
    DistillPlan p;
    p.cluster = static_cast<int32_t>(C);
    const int64_t words = tiles * kTile * kPerVec<DT> / 32;
    p.words = static_cast<int32_t>(words < kMapWords ? words : kMapWords);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.r.rows * C));
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.words) * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(C);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, distill_kernel<DT>, a, p);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int dtype, cudaStream_t s)
{
    return dtype == SV_F32 ? launch<SV_F32>(a, s) : dtype == SV_BF16 ? launch<SV_BF16>(a, s)
                                                                      : launch<SV_F16>(a, s);
}

}  // namespace svl
