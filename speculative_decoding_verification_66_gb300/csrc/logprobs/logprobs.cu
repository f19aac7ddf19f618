// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives,
// in one read of the row.
//
// Sums: lp_stream.cuh.
//
// Rank. A vector's largest element is known for the sums' sake; its elements are only
// compared with the given token's where that one reaches it, which is rare for tokens that
// a model would choose.
//
// Alternatives. The row's maxima over groups of 512 bytes (a warp's load) are kept in shared
// memory. The k-th largest of them, tau, is a lower bound of the k-th largest element; and
// the k groups that come first by (maximum, lowest index) hold all of the first k elements:
// an element of another group is behind one of each of those. So only k groups are read
// again (they are still in L2), and only elements from tau up are kept: a few more than k.
// Should they be many (ties, or a sorted row), the same argument is applied once more, to
// the vectors of 16 bytes in those groups, and leaves 8 k elements at most.
//
// A row is taken by a block, or, where there are few rows, by a cluster of up to eight, whose
// first block is told the others' sums and maxima.
//
// Bound by memory for many rows (some six to seven instructions an element).
#include "lp_finish.cuh"
#include "lp_stream.cuh"

namespace svl {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 1024;        // elements kept for the last choice: 8 SV_MAX_TOP
static_assert(kCandidates >= 8 * SV_MAX_TOP, "a vector of each of the first k");

struct LogprobPlan {
    int32_t cluster;    // blocks of a row
    int32_t groups;     // room for maxima, of groups and later of vectors
};

// The first float above x (for finite x or -inf).
__device__ __forceinline__ float next_up(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    if (b == 0x80000000u || b == 0u) return __uint_as_float(1u);
    return __uint_as_float(b & 0x80000000u ? b - 1 : b + 1);
}

// How many elements of a vector come before the token in the row's order. `last`: the token's
// place in the vector's elements (at most 0: behind it; above: before it).
template <int DT>
__device__ __noinline__ int count_ahead(uint4 v, float x_t, float above, int64_t last)
{
    uint64_t p[kPerVec<DT> / 2];
    widen<DT>(v, p);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) {
        float a, b;
        unpack2(p[i], a, b);
        n += a >= (2 * i < last ? x_t : above);
        n += b >= (2 * i + 1 < last ? x_t : above);
    }
    return n;
}

// The k that come first of n keys (larger first, then lower index), by one warp: their
// indices, rising, to `chosen`, and the last one's key.
__device__ __forceinline__ uint32_t choose(const float* keys, int32_t n, int32_t k, int32_t* chosen,
                                           int lane)
{
    // The largest value that k keys reach, bit by bit.
    uint32_t value = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t attempt = value | (1u << bit);
        int reach = 0;
        for (int32_t i = lane; i < n; i += 32) reach += ordered(keys[i]) >= attempt;
        if (__reduce_add_sync(0xFFFFFFFFu, reach) >= k) value = attempt;
    }
    int above = 0;
    for (int32_t i = lane; i < n; i += 32) above += ordered(keys[i]) > value;
    int ties = k - __reduce_add_sync(0xFFFFFFFFu, above);  // how many of the last value
    int32_t count = 0;
    for (int32_t i0 = 0; i0 < n; i0 += 32) {
        const uint32_t key = i0 + lane < n ? ordered(keys[i0 + lane]) : 0u;
        const bool equal = i0 + lane < n && key == value;
        const uint32_t eq = __ballot_sync(0xFFFFFFFFu, equal);
        const uint32_t before = (1u << lane) - 1;
        const bool take_it = key > value || (equal && __popc(eq & before) < ties);
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, take_it);
        if (take_it) chosen[count + __popc(all & before)] = i0 + lane;
        count += __popc(all);
        ties -= min(ties, __popc(eq));
    }
    return value;
}

struct Top {
    int32_t chosen[SV_MAX_TOP];
    int32_t chosen2[SV_MAX_TOP];
    unsigned long long best[kCandidates];
    int32_t count;
    uint32_t tau;
};

// Keeps the elements of a vector from tau up; called by whole warps.
template <int DT>
__device__ __forceinline__ void keep(Top& top, uint4 v, int64_t first, float tau)
{
    uint64_t p[kPerVec<DT> / 2];
    widen<DT>(v, p);
    float x[kPerVec<DT>];
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) unpack2(p[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < kPerVec<DT>; ++i) which |= (x[i] >= tau ? 1u : 0u) << i;
    if (which == 0) return;
    int at = atomicAdd(&top.count, __popc(which));
#pragma unroll
    for (int i = 0; i < kPerVec<DT>; ++i) {
        if (!(which >> i & 1)) continue;
        if (at < kCandidates)
            top.best[at] = (static_cast<unsigned long long>(ordered(x[i])) << 32) |
                           (0xFFFFFFFFu - static_cast<uint32_t>(first + i));
        ++at;
    }
}

// The first k elements, in order. `maxima`: of the row's groups; later, of vectors.
template <int DT>
__device__ __forceinline__ void alternatives(Top& top, float* maxima, const LogprobArgs& a,
                                             int32_t row, const Vecs& in, float M, double log_s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int32_t V = a.r.V, k = a.k;
    const int32_t groups = (in.n + 31) >> 5;
    const int32_t take = min(k, groups);
    if (warp == 0) {
        // Fewer groups than k: all of them, and everything in them.
        uint32_t tau = 0;
        if (groups > k)
            tau = choose(maxima, groups, k, top.chosen, lane);
        else
            for (int32_t i = lane; i < groups; i += 32) top.chosen[i] = i;
        if (lane == 0) {
            top.tau = tau;
            top.count = 0;
        }
    }
    __syncthreads();
    float tau = groups > k ? unordered(top.tau) : -inf();
    for (int32_t i = warp; i < take; i += warps) {
        const int32_t at = top.chosen[i] * 32 + lane;
        if (at < in.n) {
            // (elements around the row are -inf, and as such may be kept: not those)
            const uint4 v = ld_vec<DT>(in, at, V);
            if (tau > -inf()) keep<DT>(top, v, first_of<DT>(in, at), tau);
        }
    }
    __syncthreads();
    if (tau == -inf() || top.count > kCandidates) {
        // Too many, or no bound: the same choice among the groups' vectors.
        for (int32_t i = warp; i < take; i += warps) {
            const int32_t at = top.chosen[i] * 32 + lane;
            // (a vector beyond the row never comes before one that is not)
            maxima[i * 32 + lane] = at < in.n ? halves_max<DT>(vec_max<DT>(ld_vec<DT>(in, at, V))) : -inf();
        }
        __syncthreads();
        const int32_t vectors = take * 32, take2 = min(k, vectors);
        if (warp == 0) {
            const uint32_t value = choose(maxima, vectors, take2, top.chosen2, lane);
            if (lane == 0) {
                top.tau = value;
                top.count = 0;
            }
        }
        __syncthreads();
        tau = unordered(top.tau);
        for (int32_t i = tid; i < take2; i += blockDim.x) {
            const int32_t j = top.chosen2[i];
            const int32_t at = top.chosen[j >> 5] * 32 + (j & 31);
            if (at >= in.n) continue;
            const int64_t first = first_of<DT>(in, at);
            for (int e = 0; e < kPerVec<DT>; ++e) {
                const int64_t v = first + e;
                if (v < 0 || v >= V) continue;
                const float x = load_one<DT>(in.a0 + in.head * kElem<DT>, v);
                if (!(x >= tau) && vectors > k) continue;
                const int slot = atomicAdd(&top.count, 1);
                top.best[slot] = (static_cast<unsigned long long>(ordered(x)) << 32) |
                                 (0xFFFFFFFFu - static_cast<uint32_t>(v));
            }
        }
        __syncthreads();
    }
    // Each candidate's place is the number of those before it (none are equal).
    const int32_t n = min(top.count, kCandidates);
    for (int32_t i = tid; i < n; i += blockDim.x) {
        const unsigned long long mine = top.best[i];
        int place = 0;
        for (int32_t j = 0; j < n; ++j) place += top.best[j] > mine;
        if (place >= k) continue;
        const int64_t at = static_cast<int64_t>(row) * k + place;
        const float x = unordered(static_cast<uint32_t>(mine >> 32));
        a.top_tokens[at] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(mine));
        a.top_logprobs[at] = static_cast<float>(log_prob(x, M, a.r.c, log_s));
    }
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kMaxThreads)
    logprobs_kernel(const __grid_constant__ LogprobArgs a, const LogprobPlan plan)
{
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ RowSum part[kMaxCluster * kMaxThreads / 32];
    const int C = plan.cluster;
    const int32_t row = blockIdx.x / C, rank = blockIdx.x - row * C, V = a.r.V;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int32_t token = a.tokens == nullptr ? 0 : a.tokens[row];
    if (token == -1 || token < -1 || token >= V) {
        // (the same for all blocks of a cluster)
        if (rank != 0) return;
        const bool bad = token != -1;
        int status = bad ? SV_SEQ_BAD_TOKEN : 0;
        if (bad && a.status != nullptr) {
            // The other fault is looked for all the same.
            const uint8_t* x = row_begin(a.r.x, a.r.inner, row);
            float m = -inf();
            for (int64_t v = tid; v < V; v += blockDim.x) m = fmax_nan(m, load_one<DT>(x, v));
            const int finite = fabsf(m) < inf();
            if (__syncthreads_or(m != m || m == inf()) || !__syncthreads_or(finite))
                status |= SV_SEQ_NONFINITE;
        }
        if (tid == 0) finish_plain(a, row, bad ? kRowBad : kRowSkipped, status);
        finish_plain_top(a, row, bad ? kRowBad : kRowSkipped, tid, blockDim.x);
        return;
    }
    if (C > 1) cluster_arrive();
    const float c = a.r.c;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    float* maxima = reinterpret_cast<float*>(dynamic);
    const float x_t =
        a.tokens == nullptr ? inf() : load_one<DT>(in.a0 + in.head * kElem<DT>, token);
    const float above = next_up(x_t);
    const float step = 16.f / c;
    const float low = lowest_of<DT>(c);
    Running st;
    start(st);
    int32_t ahead = 0;
    const int32_t tiles = tiles_of(in.n);
    for (int32_t tile = rank * warps + warp; tile < tiles; tile += C * warps) {
        const int32_t base = tile * kTile;
        uint4 v[kInFlight];
        ld_tile<DT>(v, in, base, lane, V);
        float top;
        if (TOP) {
            float tops[kInFlight], groups[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                tops[u] = halves_max<DT>(vec_max<DT>(v[u]));
                groups[u] = warp_max(tops[u]);
            }
            if (lane == 0)
                reinterpret_cast<float4*>(maxima)[tile] =
                    make_float4(groups[0], groups[1], groups[2], groups[3]);
            top = fmax_nan(fmax_nan(tops[0], tops[1]), fmax_nan(tops[2], tops[3]));
        } else {
            uint32_t t = vec_max<DT>(v[0]);
#pragma unroll
            for (int u = 1; u < kInFlight; ++u) t = packed_max<DT>(t, vec_max<DT>(v[u]));
            top = halves_max<DT>(t);
        }
        if (top >= x_t) {
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (halves_max<DT>(vec_max<DT>(v[u])) >= x_t)
                    ahead += count_ahead<DT>(v[u], x_t, above,
                                             token - first_of<DT>(in, base + lane + u * 32));
        }
        take<DT, true>(st, v, top, c, step, low);
    }
    const RowSum mine = warp_join(st, ahead, c);
    if (C == 1) {
        if (lane == 0) part[warp] = mine;
        __syncthreads();
    } else {
        cluster_wait();
        if (lane == 0) {
            const RowSum* slot = &part[rank * warps + warp];
            st_cluster(&slot->m, 0, mine.m);
            st_cluster(&slot->s, 0, mine.s);
            st_cluster(&slot->e, 0, mine.e);
            st_cluster(&slot->ahead, 0, __int_as_float(mine.ahead));
        }
        if (TOP && rank != 0) {
            // This block's maxima, those that its own warps wrote among them.
            __syncthreads();
            for (int32_t t0 = rank * warps; t0 < tiles; t0 += C * warps)
                for (int32_t g = t0 * kInFlight + tid; g < min(t0 + warps, tiles) * kInFlight;
                     g += blockDim.x)
                    st_cluster(&maxima[g], 0, maxima[g]);
        }
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
    }
    RowSum all = part[0];
    for (int w = 1; w < warps * C; ++w) all = join(all, part[w], c);
    if (!(fabsf(all.m) < inf())) {
        if (tid == 0) finish_plain(a, row, kRowBad, SV_SEQ_NONFINITE);
        finish_plain_top(a, row, kRowBad, tid, blockDim.x);
        return;
    }
    const double log_s = log_wide(all.s);
    if (tid == 0) {
        // (the -inf that stand for what is before the row were counted as ties of a masked token)
        const int ahead = all.ahead - (x_t == -inf() ? in.head : 0);
        finish_row(a, row, all.m, all.s, all.e, x_t, ahead, log_s);
    }
    if (TOP)
        alternatives<DT>(*reinterpret_cast<Top*>(dynamic + static_cast<size_t>(plan.groups) * 4),
                         maxima, a, row, in, all.m, log_s);
}

template <int DT, bool TOP>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s)
{
    constexpr int64_t kBlocks = 304;
    const int64_t tiles = tiles_of((a.r.V + kPerVec<DT> - 1) / kPerVec<DT> + 1);
    int warps = 1;
    while (warps * 32 < kMaxThreads && warps < tiles) warps *= 2;
    // A cluster where there are fewer rows than two blocks an SM, and a turn for each block.
    int64_t C = 1;
    while (C < kMaxCluster && a.r.rows * C < kBlocks && tiles > C * warps) C *= 2;
    LogprobPlan p;
    p.cluster = static_cast<int32_t>(C);
    // Maxima of groups, and of the chosen groups' vectors.
    const int64_t groups = tiles * kInFlight;
    const int64_t again = 32 * (a.k < groups ? a.k : groups);
    p.groups = static_cast<int32_t>(groups > again ? groups : again);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.r.rows * C));
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = TOP ? p.groups * 4 + sizeof(Top) : 0;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(C);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, TOP>, a, p);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, cudaStream_t s)
{
    const bool top = a.k > 0;
    if (dtype == SV_F32) return top ? launch<SV_F32, true>(a, s) : launch<SV_F32, false>(a, s);
    if (dtype == SV_BF16) return top ? launch<SV_BF16, true>(a, s) : launch<SV_BF16, false>(a, s);
    return top ? launch<SV_F16, true>(a, s) : launch<SV_F16, false>(a, s);
}

}  // namespace svl
