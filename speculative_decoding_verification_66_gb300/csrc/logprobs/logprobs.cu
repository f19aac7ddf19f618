// logprobs.cu -- log probabilities of given tokens, entropy and top alternatives,
// in one read of the row.
//
// Sums: lp_stream.cuh.
//
// Rank. A turn's largest element is known for the sums' sake; its elements are only compared
// with the given token's where that one reaches it, a pair of 16-bit ones at a time. (One by
// one, in the vectors that reach it: 85 us for 1024 rows of 128256 whose tokens have some 800
// before them.)
//
// Alternatives. The row's maxima over groups of 512 bytes (a warp's load) are kept in shared
// memory. The k-th largest of them, tau, is a lower bound of the k-th largest element; and
// the k groups that come first by (maximum, lowest index) hold all of the first k elements:
// an element of another group is behind one of each of those. So only k groups are read
// again (they are still in L2), and only elements from tau up are kept: a few more than k.
// Should they be many (ties, or a sorted row), the same argument is applied once more, to
// the vectors of 16 bytes in those groups, and leaves 8 k elements at most.
//
// A row is cut into pieces of up to 64 KB, a block each: many small blocks load the memory
// evenly to the end, and one row alone is read by thirty SMs. A piece leaves its sums and its
// groups' maxima in the workspace; the block that is the last of its row to do so (a counter a
// row, which starts at 0 and is 0 again afterwards) finishes the row while others read on.
// Pieces are joined in order, so that who is last makes no difference.
//
// Bound by memory for many rows (some six to seven instructions an element).
#include "lp_finish.cuh"
#include "lp_stream.cuh"

namespace svl {
namespace {

constexpr int kMaxWarps = 4;

struct LogprobPlan {
    int32_t pieces;      // of a row, a block each
    int32_t piece;       // warps' turns in a piece
    int32_t groups;      // maxima of a row (a multiple of 4)
    int32_t keys;        // room for them, and for those of the chosen groups' vectors
    int32_t candidates;  // elements kept for the last choice: a vector of each of the first k,
                         // at least
    Split split;         // with more than one piece
};

// Numbers of the logits' type as words that hold one or two of them, and the next one up
// (from a finite one or -inf).
template <int DT>
__device__ __forceinline__ uint32_t next_up(uint32_t w)
{
    if (DT == SV_F32) return (w << 1) == 0 ? 1u : w & 0x80000000u ? w - 1 : w + 1;
    const uint32_t h = w & 0xFFFFu;
    const uint32_t up = (h & 0x7FFFu) == 0 ? 1u : h & 0x8000u ? h - 1 : h + 1;
    return up | up << 16;
}

// How many elements of a lane's vectors reach a bound.
template <int DT>
__device__ __forceinline__ int32_t count_from(const uint4 (&v)[kInFlight], uint32_t bound)
{
    int32_t n = 0;
    uint32_t acc = 0;
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (DT == SV_F32) {
                n += __uint_as_float(w[i]) >= __uint_as_float(bound);
            } else if (DT == SV_BF16) {
                acc -= __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                   *reinterpret_cast<const __nv_bfloat162*>(&bound));
            } else {
                acc -= __hge2_mask(*reinterpret_cast<const __half2*>(&w[i]),
                                   *reinterpret_cast<const __half2*>(&bound));
            }
        }
    }
    // A low half's mask of ones takes 2^16 - 1 off, a high one's adds 2^16:
    // acc = 2^16 (high - low) + low.
    if (DT != SV_F32) n = (static_cast<int32_t>(acc) >> 16) + 2 * static_cast<int32_t>(acc & 0xFFFFu);
    return n;
}

// The same where the token is among the warp's vectors: those before it count if they are as
// large, those behind it only if they are larger. `at`: the token's place, counted from the
// vector's first element.
template <int DT>
__device__ __noinline__ int32_t count_around(uint4 v, float x_t, float above, int64_t at)
{
    uint64_t p[kPerVec<DT> / 2];
    widen<DT>(v, p);
    int32_t n = 0;
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) {
        float a, b;
        unpack2(p[i], a, b);
        n += a >= (2 * i < at ? x_t : above);
        n += b >= (2 * i + 1 < at ? x_t : above);
    }
    return n;
}

// Bits of an ordered key (of a number of the logits' type) that are all zeros or all ones.
template <int DT>
constexpr int kIdleBits = DT == SV_F32 ? 0 : DT == SV_BF16 ? 16 : 13;

// The k that come first of n ordered keys (larger first, then lower index), by one warp:
// their indices, rising, to `chosen`, and the last one's key. n: a multiple of 128, or keys
// beyond it up to one that are 0.
template <int DT>
__device__ __forceinline__ uint32_t choose(const uint32_t* keys, int32_t n, int32_t k,
                                           int32_t* chosen, int lane)
{
    const uint4* four = reinterpret_cast<const uint4*>(keys);
    const int32_t fours = (n + 3) >> 2;
    // The largest value that k keys reach, bit by bit.
    uint32_t value = 0;
    for (int bit = 31; bit >= kIdleBits<DT>; --bit) {
        const uint32_t attempt = value | (1u << bit);
        int reach = 0;
        for (int32_t i = lane; i < fours; i += 32) {
            const uint4 q = four[i];
            reach += (q.x >= attempt) + (q.y >= attempt) + (q.z >= attempt) + (q.w >= attempt);
        }
        if (__reduce_add_sync(0xFFFFFFFFu, reach) >= k) value = attempt;
    }
    if (kIdleBits<DT> > 0 && !(value & 0x80000000u)) value |= (1u << kIdleBits<DT>) - 1;
    int above = 0;
    for (int32_t i = lane; i < fours; i += 32) {
        const uint4 q = four[i];
        above += (q.x > value) + (q.y > value) + (q.z > value) + (q.w > value);
    }
    int ties = k - __reduce_add_sync(0xFFFFFFFFu, above);  // how many of the last value
    int32_t count = 0;
    const uint32_t before = (1u << lane) - 1;
    for (int32_t i0 = 0; i0 < n && count < k; i0 += 32) {
        const uint32_t key = i0 + lane < n ? keys[i0 + lane] : 0u;
        const bool equal = key == value;  // (no key is 0)
        const uint32_t eq = __ballot_sync(0xFFFFFFFFu, equal);
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
    int32_t count;
    uint32_t tau;
    uint32_t flags;
    int32_t candidates;          // room in best
    unsigned long long* best;    // key, and the index's complement
};

// Keeps the elements of a vector from tau up.
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
        if (at < top.candidates)
            top.best[at] = (static_cast<unsigned long long>(ordered(x[i])) << 32) |
                           (0xFFFFFFFFu - static_cast<uint32_t>(first + i));
        ++at;
    }
}

// The first k elements, in order. `maxima`: of the row's groups; `keys`: room for them (the same,
// perhaps), and for those of the chosen groups' vectors. (SPLIT: other blocks wrote the maxima.)
template <int DT, bool SPLIT>
__device__ __forceinline__ void alternatives(Top& top, const float* maxima,
                                             uint32_t* keys, const LogprobArgs& a, int32_t row,
                                             const Vecs& in, float M, double log_s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int32_t V = a.r.V, k = a.k;
    const int32_t groups = (in.n + 31) >> 5;
    const int32_t take = min(k, groups);
    for (int32_t i = tid; i < ((groups + 3) & ~3); i += blockDim.x)
        keys[i] = i < groups ? ordered(SPLIT ? __ldcg(maxima + i) : maxima[i]) : 0u;
    __syncthreads();
    if (warp == 0) {
        // Fewer groups than k: all of them, and everything in them.
        uint32_t tau = 0;
        if (groups > k)
            tau = choose<DT>(keys, groups, k, top.chosen, lane);
        else
            for (int32_t i = lane; i < groups; i += 32) top.chosen[i] = i;
        if (lane == 0) {
            top.tau = tau;
            top.count = 0;
        }
    }
    __syncthreads();
    float tau = groups > k ? unordered(top.tau) : -inf();
    if (tau > -inf()) {
        for (int32_t i0 = warp; i0 < take; i0 += kInFlight * warps) {
            uint4 v[kInFlight];
            int32_t at[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int32_t i = i0 + u * warps;
                at[u] = i < take ? top.chosen[i] * 32 + lane : in.n;
                v[u] = ld_vec<DT>(in, at[u], V);
            }
            // (what stands around the row is -inf, and below tau)
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) keep<DT>(top, v[u], first_of<DT>(in, at[u]), tau);
        }
    }
    __syncthreads();
    if (tau == -inf() || top.count > top.candidates) {
        // Too many, or no bound: the same choice among the groups' vectors.
        for (int32_t i = warp; i < take; i += warps) {
            const int32_t at = top.chosen[i] * 32 + lane;
            // (a vector beyond the row never comes before one that is not)
            keys[i * 32 + lane] = ordered(
                at < in.n ? halves_max<DT>(vec_max<DT>(ld_vec<DT>(in, at, V))) : -inf());
        }
        __syncthreads();
        const int32_t vectors = take * 32, take2 = min(k, vectors);
        if (warp == 0) {
            const uint32_t value = choose<DT>(keys, vectors, take2, top.chosen2, lane);
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
    const int32_t n = min(top.count, top.candidates);
    for (int32_t i = tid; i < n; i += blockDim.x) {
        const unsigned long long mine = top.best[i];
        int place = 0;
#pragma unroll 4
        for (int32_t j = 0; j < n; ++j) place += top.best[j] > mine;
        if (place >= k) continue;
        const int64_t at = static_cast<int64_t>(row) * k + place;
        const float x = unordered(static_cast<uint32_t>(mine >> 32));
        a.top_tokens[at] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(mine));
        a.top_logprobs[at] = static_cast<float>(log_prob(x, M, a.r.c, log_s));
    }
}

// A row that a group of threads finds nothing asked of, or a bad token.
template <int DT>
__device__ __forceinline__ void finish_other(const LogprobArgs& a, int32_t row,
                                             int32_t token, uint32_t* flags)
{
    const bool bad = token != -1;
    int status = bad ? SV_SEQ_BAD_TOKEN : 0;
    if (bad && a.status != nullptr) {
        // The other fault is looked for all the same.
        const uint8_t* x = row_begin(a.r.x, a.r.inner, row);
        float m = -inf();
        for (int64_t v = threadIdx.x; v < a.r.V; v += blockDim.x) m = fmax_nan(m, load_one<DT>(x, v));
        if (threadIdx.x == 0) *flags = 0;
        __syncthreads();
        atomicOr(flags, (m != m || m == inf() ? 2u : 0u) | (fabsf(m) < inf() ? 1u : 0u));
        __syncthreads();
        if (*flags != 1u) status |= SV_SEQ_NONFINITE;
        __syncthreads();
    }
    const int kind = bad ? kRowBad : kRowSkipped;
    if (threadIdx.x == 0) finish_plain(a, row, kind, status);
    finish_plain_top(a, row, kind, threadIdx.x, blockDim.x);
}

// A row's results from its sums.
template <int DT, bool TOP, bool SPLIT>
__device__ __forceinline__ void finish_all(const LogprobArgs& a, int32_t row,
                                           const Vecs& in, const RowSum& all, float x_t, Top& top,
                                           const float* maxima, uint32_t* keys)
{
    if (!(fabsf(all.m) < inf())) {
        if (threadIdx.x == 0) finish_plain(a, row, kRowBad, SV_SEQ_NONFINITE);
        finish_plain_top(a, row, kRowBad, threadIdx.x, blockDim.x);
        return;
    }
    const double log_s = log_wide(all.s);
    if (threadIdx.x == 0) {
        // (the -inf that stand for what is before the row were counted as ties of a masked token)
        const int ahead = all.ahead - (x_t == -inf() ? in.head : 0);
        finish_row(a, row, all.m, all.s, all.e, x_t, ahead, log_s);
    }
    if (TOP) alternatives<DT, SPLIT>(top, maxima, keys, a, row, in, all.m, log_s);
}

// What the token of a row asks of its elements.
struct Asked {
    float x_t;                    // its logit; +inf: no token, nothing is counted
    uint32_t at_least, beyond;    // bounds before and behind it
    int32_t token, tile;          // and the turn that it is in
};

template <int DT>
__device__ __forceinline__ Asked asked_of(const LogprobArgs& a, const Vecs& in, int32_t token)
{
    Asked q;
    q.token = token;
    q.x_t = a.tokens == nullptr ? inf() : load_one<DT>(in.a0 + in.head * kElem<DT>, token);
    q.at_least = pair_of<DT>(q.x_t);
    q.beyond = next_up<DT>(q.at_least);
    q.tile = a.tokens == nullptr ? -1
                                 : static_cast<int32_t>((static_cast<int64_t>(token) + in.head) /
                                                        (kPerVec<DT> * kTile));
    return q;
}

// One turn of a row.
template <int DT, bool TOP>
__device__ __forceinline__ void do_tile(Running& st, int32_t& ahead, const uint4 (&v)[kInFlight],
                                        int32_t tile, int32_t head, const Asked& q,
                                        float* maxima, float c, float step, float low, int lane)
{
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
    if (tile == q.tile) {
        const float above = halves_max<DT>(q.beyond);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            ahead += count_around<DT>(v[u], q.x_t, above,
                                      q.token + head - static_cast<int64_t>(tile * kTile + lane + u * 32) * kPerVec<DT>);
    } else if (__any_sync(0xFFFFFFFFu, top >= q.x_t)) {
        ahead += count_from<DT>(v, tile < q.tile ? q.at_least : q.beyond);
    }
    take<DT, true>(st, v, top, c, step, low);
}

// A piece of a row to a block. SPLIT: of several.
template <int DT, bool TOP, bool SPLIT>
__global__ void __launch_bounds__(kMaxWarps * 32, 10)
    logprobs_kernel(const __grid_constant__ LogprobArgs a, const __grid_constant__ LogprobPlan plan)
{
    // Keys, then candidates.
    extern __shared__ __align__(16) uint32_t dynamic[];
    __shared__ RowSum part[kMaxWarps];
    __shared__ Top top;
    const int32_t row = SPLIT ? blockIdx.x / plan.pieces : blockIdx.x;
    const int32_t piece = SPLIT ? blockIdx.x - row * plan.pieces : 0, V = a.r.V;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int32_t token = a.tokens == nullptr ? 0 : a.tokens[row];
    if (token < 0 || token >= V) {
        if (piece == 0) finish_other<DT>(a, row, token, &top.flags);
        return;
    }
    const float c = a.r.c;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    float* maxima = !TOP    ? nullptr
                    : SPLIT ? plan.split.maxima + static_cast<int64_t>(row) * plan.groups
                            : reinterpret_cast<float*>(dynamic);
    const Asked q = asked_of<DT>(a, in, token);
    const float step = 16.f / c, low = lowest_of<DT>(c);
    Running st;
    start(st);
    int32_t ahead = 0;
    const int32_t tiles = tiles_of(in.n);
    const int32_t first = SPLIT ? piece * plan.piece : 0;
    const int32_t end = SPLIT ? min(first + plan.piece, tiles) : tiles;
    for (int32_t tile = first + warp; tile < end; tile += warps) {
        uint4 v[kInFlight];
        ld_tile<DT>(v, in, tile * kTile, lane, V);
        do_tile<DT, TOP>(st, ahead, v, tile, in.head, q, maxima, c, step, low, lane);
    }
    const RowSum mine = warp_join(st, ahead, c);
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    RowSum all = part[0];
    for (int w = 1; w < warps; ++w) all = join(all, part[w], c);
    if (SPLIT) {
        if (!last_piece(plan.split, row, piece, plan.pieces, all, &top.flags)) return;
        all = join_pieces(plan.split, row, plan.pieces, c, lane);
    }
    if (TOP) {
        if (tid == 0) {
            top.best = reinterpret_cast<unsigned long long*>(dynamic + plan.keys);
            top.candidates = plan.candidates;
        }
        __syncthreads();
    }
    finish_all<DT, TOP, SPLIT>(a, row, in, all, q.x_t, top, maxima, dynamic);
}

template <int DT>
LogprobPlan plan_of(const Rows& r, int32_t k, int* warps)
{
    LogprobPlan p{};
    const int32_t tiles = tiles_of((static_cast<int64_t>(r.V) + kPerVec<DT> - 1) / kPerVec<DT> + 1);
    p.pieces = pieces_of(r.rows, tiles, kMaxWarps, &p.piece);
    *warps = 1;
    while (*warps < kMaxWarps && *warps < p.piece) *warps *= 2;
    p.groups = tiles * kInFlight;
    const int32_t vectors = 32 * (k < p.groups ? k : p.groups);
    p.keys = p.groups > vectors ? p.groups : vectors;
    p.candidates = 8 * k > 512 ? 8 * k : 512;
    return p;
}

template <int DT, bool TOP>
cudaError_t launch(const LogprobArgs& a, void* workspace, cudaStream_t s)
{
    int warps = 1;
    LogprobPlan p = plan_of<DT>(a.r, a.k, &warps);
    if (p.pieces > 1) p.split = split_of(workspace, a.r.rows, p.pieces);
    const size_t bytes = TOP ? p.keys * 4 + p.candidates * 8 : 0;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.pieces) * a.r.rows);
    const auto k = p.pieces > 1 ? logprobs_kernel<DT, TOP, true> : logprobs_kernel<DT, TOP, false>;
    if (bytes > 45000) {  // (beside the static part, more than is allowed unasked)
        const cudaError_t e =
            cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
        if (e != cudaSuccess) return e;
    }
    k<<<grid, warps * 32, bytes, s>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

size_t logprobs_workspace(const Rows& r, int dtype, int32_t k)
{
    int warps;
    const LogprobPlan p = dtype == SV_F32 ? plan_of<SV_F32>(r, k, &warps)
                                          : plan_of<SV_BF16>(r, k, &warps);
    return p.pieces > 1 ? split_bytes(r.rows, p.pieces, k > 0 ? p.groups : 0) : 0;
}

cudaError_t launch_logprobs(const LogprobArgs& a, int dtype, void* workspace, cudaStream_t s)
{
    const bool top = a.k > 0;
    if (dtype == SV_F32)
        return top ? launch<SV_F32, true>(a, workspace, s) : launch<SV_F32, false>(a, workspace, s);
    if (dtype == SV_BF16)
        return top ? launch<SV_BF16, true>(a, workspace, s) : launch<SV_BF16, false>(a, workspace, s);
    return top ? launch<SV_F16, true>(a, workspace, s) : launch<SV_F16, false>(a, workspace, s);
}

}  // namespace svl
