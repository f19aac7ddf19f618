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
// Few rows are cut into pieces, a block each (cut_of; one row of 128256 bfloat16 is read by
// eleven SMs, or by three with alternatives). A piece leaves its sums and its groups' maxima in the
// workspace; the block that is the last of its row to do so (a counter a row, which starts at 0 and
// is 0 again afterwards) finishes the row while others read on. Pieces are joined in order, so that
// who is last makes no difference.
//
// Bound by memory for many rows: half of the issue slots are taken (some six to seven instructions
// an element). 1024 rows of 128256 bfloat16, 263 MB: 51 us without alternatives, 61 with 20, 80
// with 128 (a block's choice and order of 128 is not hidden where all rows make one wave); 4096
// rows 172, 217 and 291: 6.1, 4.8 and 3.6 TB/s. A plain sum over the 263 MB takes 49.
#include "lp_finish.cuh"
#include "lp_stream.cuh"

namespace svl {
namespace {

struct LogprobPlan {
    Cut cut;
    int32_t groups;      // maxima of a row (a multiple of 4)
    int32_t keys;        // room for them, and for those of the chosen groups' vectors
    int32_t candidates;  // elements kept for the last choice: a vector of each of the first k,
                         // at least
    Split split;         // where rows are cut
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

// What a block's threads share while they choose.
struct Choice {
    uint32_t bins[256];
    uint32_t digit, need;
    int32_t over[kMostWarps], ties[kMostWarps];
};

// The k that come first of n ordered keys (larger first, then lower index; n > 0, no key is 0):
// their indices, rising, to `chosen`; returns the last one's key. By all threads of a block,
// digit by digit of eight bits: a histogram of the keys that agree with the k-th so far, then
// its next digit. (Bit by bit, by one warp: 9.6 us for 504 keys, this 2.5.)
template <int DT>
__device__ __forceinline__ uint32_t choose(const uint32_t* keys, int32_t n, int32_t k, int32_t* chosen,
                                           Choice& ch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    uint32_t value = 0, mask = 0;
    int32_t need = k;
#pragma unroll 1
    for (int shift = 24; shift + 8 > kIdleBits<DT>; shift -= 8) {
        for (int b = tid; b < 256; b += blockDim.x) ch.bins[b] = 0u;
        __syncthreads();
        for (int32_t i = tid; i < n; i += blockDim.x) {
            const uint32_t key = keys[i];
            if ((key & mask) == value) atomicAdd(&ch.bins[key >> shift & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // Eight bins a lane, from the top.
            uint32_t mine[8], sum = 0;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                mine[b] = ch.bins[255 - 8 * lane - b];
                sum += mine[b];
            }
            uint32_t upto = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
                if (lane >= off) upto += o;
            }
            uint32_t before = upto - sum;
            if (before < static_cast<uint32_t>(need) && upto >= static_cast<uint32_t>(need)) {
                int digit = -1;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    if (digit < 0 && before + mine[b] >= static_cast<uint32_t>(need))
                        digit = 255 - 8 * lane - b;
                    if (digit < 0) before += mine[b];
                }
                ch.digit = digit;
                ch.need = need - before;
            }
        }
        __syncthreads();
        value |= ch.digit << shift;
        need = ch.need;
        mask |= 255u << shift;
    }
    if (kIdleBits<DT> > 0) value |= value & 0x80000000u ? 0u : (1u << kIdleBits<DT>) - 1;
    // Each warp has a range of the keys: how many it takes, then where they go.
    const int32_t per = ((n + warps * 32 - 1) / (warps * 32)) * 32;
    const int32_t lo = warp * per, hi = min(lo + per, n);
    int32_t over = 0, ties = 0;
    for (int32_t i0 = lo; i0 < hi; i0 += 32) {
        const uint32_t key = i0 + lane < hi ? keys[i0 + lane] : 0u;
        over += __popc(__ballot_sync(0xFFFFFFFFu, key > value));
        ties += __popc(__ballot_sync(0xFFFFFFFFu, key == value));
    }
    if (lane == 0) {
        ch.over[warp] = over;
        ch.ties[warp] = ties;
    }
    __syncthreads();
    int32_t to = 0, left = need;  // ties that are taken, from here on
    for (int w = 0; w < warp; ++w) {
        to += ch.over[w] + min(ch.ties[w], left);
        left -= min(ch.ties[w], left);
    }
    const uint32_t before = (1u << lane) - 1;
    for (int32_t i0 = lo; i0 < hi; i0 += 32) {
        const uint32_t key = i0 + lane < hi ? keys[i0 + lane] : 0u;
        const uint32_t equal = __ballot_sync(0xFFFFFFFFu, key == value);
        const bool mine = key > value || (key == value && __popc(equal & before) < left);
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, mine);
        if (mine) chosen[to + __popc(all & before)] = i0 + lane;
        to += __popc(all);
        left -= min(left, __popc(equal));
    }
    __syncthreads();
    return value;
}

struct Top {
    int32_t chosen[SV_MAX_TOP];
    int32_t chosen2[SV_MAX_TOP];
    int32_t count, vectors;
    uint32_t flags;
    Choice choice;
    int32_t candidates;          // room in best
    unsigned long long* best;    // key, and the index's complement
};

// The elements of a vector from tau up, a bit for each.
template <int DT>
__device__ __forceinline__ uint32_t reach(uint4 v, float tau)
{
    uint64_t p[kPerVec<DT> / 2];
    widen<DT>(v, p);
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) {
        float a, b;
        unpack2(p[i], a, b);
        which |= (a >= tau ? 1u : 0u) << (2 * i) | (b >= tau ? 2u : 0u) << (2 * i);
    }
    return which;
}

// Keeps them, from place `at` on.
template <int DT>
__device__ __forceinline__ void keep(Top& top, uint4 v, uint32_t which, int64_t first, int at)
{
    uint64_t p[kPerVec<DT> / 2];
    widen<DT>(v, p);
    for (; which != 0; which &= which - 1, ++at) {
        const int i = __ffs(which) - 1;
        uint64_t two = p[0];
#pragma unroll
        for (int q = 1; q < kPerVec<DT> / 2; ++q)
            if (i >> 1 == q) two = p[q];
        float a, b;
        unpack2(two, a, b);
        if (at < top.candidates)
            top.best[at] = (static_cast<unsigned long long>(ordered(i & 1 ? b : a)) << 32) |
                           (0xFFFFFFFFu - static_cast<uint32_t>(first + i));
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
    if (tid == 0) top.count = top.vectors = 0;
    __syncthreads();
    float tau = -inf();
    if (groups > k) {
        tau = unordered(choose<DT>(keys, groups, k, top.chosen, top.choice));
    } else {
        // Fewer groups than k: all of them, and everything in them.
        for (int32_t i = tid; i < groups; i += blockDim.x) top.chosen[i] = i;
        __syncthreads();
    }
    if (tau > -inf()) {
        constexpr int kBatch = 8;
        for (int32_t i0 = warp; i0 < take; i0 += kBatch * warps) {
            // (whole groups without a case between the loads, or each would wait for the last)
            uint4 v[kBatch];
            bool inside = true;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int32_t base = top.chosen[min(i0 + u * warps, take - 1)] * 32;
                inside &= base >= in.full && base + 32 <= in.full_end;
            }
            if (inside) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    v[u] = ld_stream(in.a0 + static_cast<int64_t>(
                                                 top.chosen[min(i0 + u * warps, take - 1)] * 32 + lane) * 16);
            } else {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    v[u] = ld_vec<DT>(in, top.chosen[min(i0 + u * warps, take - 1)] * 32 + lane, V);
            }
            // The vectors that reach tau, listed where the keys were (there is room for all).
            uint32_t hit[kBatch], sum = 0;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const bool reaches = halves_max<DT>(vec_max<DT>(v[u])) >= tau;
                hit[u] = i0 + u * warps < take ? __ballot_sync(0xFFFFFFFFu, reaches) : 0u;
                sum += __popc(hit[u]);
            }
            int32_t at = 0;
            if (lane == 0) at = atomicAdd(&top.vectors, sum);
            at = __shfl_sync(0xFFFFFFFFu, at, 0);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (hit[u] >> lane & 1)
                    keys[at + __popc(hit[u] & ((1u << lane) - 1))] =
                        top.chosen[i0 + u * warps] * 32 + lane;
                at += __popc(hit[u]);
            }
        }
        __syncthreads();
        // Their elements, a thread a vector. (What stands around the row is -inf, and below tau.)
        for (int32_t i = tid; i < top.vectors; i += blockDim.x) {
            const int32_t vec = keys[i];
            const uint4 v = ld_vec<DT>(in, vec, V);
            const uint32_t which = reach<DT>(v, tau);
            keep<DT>(top, v, which, first_of<DT>(in, vec), atomicAdd(&top.count, __popc(which)));
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
        if (tid == 0) top.count = 0;
        tau = unordered(choose<DT>(keys, vectors, take2, top.chosen2, top.choice));
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
    // Each candidate's place is the number of those before it (none are equal): a thread has
    // two at a time, and all others go by, two at a time.
    const int32_t n = min(top.count, top.candidates);
    if (tid == 0 && (n & 1)) top.best[n] = 0ull;  // (room for one more: candidates is even)
    __syncthreads();
    constexpr int kMine = 2;
    const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(top.best);
    for (int32_t i0 = tid; i0 < n; i0 += kMine * blockDim.x) {
        unsigned long long mine[kMine];
        int place[kMine];
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int32_t i = i0 + u * blockDim.x;
            mine[u] = i < n ? top.best[i] : ~0ull;
            place[u] = 0;
        }
#pragma unroll 4
        for (int32_t j = 0; j < (n + 1) >> 1; ++j) {
            const ulonglong2 two = pairs[j];
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                place[u] += two.x > mine[u];
                place[u] += two.y > mine[u];
            }
        }
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            if (i0 + u * blockDim.x >= n || place[u] >= k) continue;
            const int64_t at = static_cast<int64_t>(row) * k + place[u];
            const float x = unordered(static_cast<uint32_t>(mine[u] >> 32));
            a.top_tokens[at] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(mine[u]));
            a.top_logprobs[at] = static_cast<float>(log_prob(x, M, a.r.c, log_s));
        }
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
    if (TOP) alternatives<DT, SPLIT>(top, maxima, keys, a, row, in, all.m, log_s);
    if (threadIdx.x == blockDim.x - 32) {  // (the last warp has the fewest alternatives)
        // (the -inf that stand for what is before the row were counted as ties of a masked token)
        const int ahead = all.ahead - (x_t == -inf() ? in.head : 0);
        finish_row(a, row, all.m, all.s, all.e, x_t, ahead, log_s);
    }
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
__global__ void __launch_bounds__((TOP ? kMostWarps : kLeastWarps) * 32, TOP ? 2 : 8)
    logprobs_kernel(const __grid_constant__ LogprobArgs a, const __grid_constant__ LogprobPlan plan)
{
    // Keys, then candidates.
    extern __shared__ __align__(16) uint32_t dynamic[];
    __shared__ RowSum part[TOP ? kMostWarps : kLeastWarps];
    __shared__ Top top;
    const int32_t row = SPLIT ? row_of(plan.cut, blockIdx.x) : blockIdx.x, V = a.r.V;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int32_t token = a.tokens == nullptr ? 0 : a.tokens[row];
    if (token < 0 || token >= V) {
        if (!SPLIT || part_of(plan.cut, blockIdx.x, row, 0).piece == 0)
            finish_other<DT>(a, row, token, &top.flags);
        return;
    }
    const float c = a.r.c;
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    float* maxima = !TOP    ? nullptr
                    : SPLIT ? plan.split.maxima + static_cast<int64_t>(row - plan.cut.whole) * plan.groups
                            : reinterpret_cast<float*>(dynamic);
    const Asked q = asked_of<DT>(a, in, token);
    const float step = kBehindEntropy / c, low = lowest_of<DT>(c);
    Running st;
    start(st);
    int32_t ahead = 0;
    const int32_t tiles = tiles_of(in.n);
    const Part mine = SPLIT ? part_of(plan.cut, blockIdx.x, row, tiles) : Part{row, 0, 1, 0, tiles};
    for (int32_t tile = mine.first + warp; tile < mine.end; tile += warps) {
        uint4 v[kInFlight];
        ld_tile<DT>(v, in, tile * kTile, lane, V);
        do_tile<DT, TOP>(st, ahead, v, tile, in.head, q, maxima, c, step, low, lane);
    }
    RowSum all = block_join(part, warp_join(st, ahead, c), c);
    if (SPLIT && mine.pieces > 1) {
        if (!last_piece(plan.split, row - plan.cut.whole, mine, all, &top.flags)) return;
        all = join_pieces(plan.split, row - plan.cut.whole, mine.pieces, c, lane);
    } else {
        if (tid == 0) part[0] = all;
        __syncthreads();
        all = part[0];
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

// Keys and candidates of the longest row and of most alternatives have room beside the static part
// in what a block gets unasked.
constexpr int32_t kMostGroups = ((SV_MAX_TOP_VOCAB + 3) / 4 + 1 + kTile - 1) / kTile * kInFlight;
static_assert(32 * SV_MAX_TOP <= kMostGroups, "the groups' maxima are the most keys");
static_assert(kMostGroups * 4 + 8 * SV_MAX_TOP * 8 + sizeof(Top) + kMostWarps * sizeof(RowSum) <= 49152,
              "else the kernel has to be allowed more");

template <int DT>
LogprobPlan plan_of(const Rows& r, int32_t k, int* warps)
{
    LogprobPlan p{};
    const int32_t tiles = most_tiles(r.V, kPerVec<DT>);
    // (alternatives, 128 of 128256 bfloat16: with 4, 8 and 16 warps 40 rows 29, 23 and 21 us, 304 rows
    // 49, 39 and 33, 608 rows 66, 49 and 74, 912 rows 72, 88 and 100; 20 of them 20, 18, 18, 31, 31,
    // 29, 45, 41, 66, 57, 72, 89; none 12, 12, 14, 23, 24, 23, 37, 35, 47, 49, 55, 64)
    const int most = k > 0 ? warps_of(r.rows) : kLeastWarps;
    p.cut = cut_of(r.rows, tiles, most, k > 0);
    *warps = 1;
    while (*warps < most && *warps < p.cut.piece) *warps *= 2;
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
    const bool cut = p.cut.pieces > 1;
    if (cut) p.split = split_of(workspace, a.r.rows - p.cut.whole, p.cut.pieces);
    const size_t bytes = TOP ? p.keys * 4 + p.candidates * 8 : 0;
    const unsigned grid = static_cast<unsigned>(blocks_of(p.cut, a.r.rows));
    const auto k = cut ? logprobs_kernel<DT, TOP, true> : logprobs_kernel<DT, TOP, false>;
    k<<<grid, warps * 32, bytes, s>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

size_t logprobs_workspace(const Rows& r, int dtype, int32_t k)
{
    int warps;
    const LogprobPlan p = dtype == SV_F32 ? plan_of<SV_F32>(r, k, &warps)
                                          : plan_of<SV_BF16>(r, k, &warps);
    return p.cut.pieces > 1 ? split_bytes(r.rows - p.cut.whole, p.cut.pieces, k > 0 ? p.groups : 0) : 0;
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
