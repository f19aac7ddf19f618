// distill.cu -- divergence of a teacher's entries from rows of logits, and what its
// gradient needs (rows_grad.cu has that).
//
// With SV_TAIL_BUCKET the sum over the tokens without entries must not be a difference:
// where a teacher's few tokens have nearly all of the student's probability too, nothing
// would be left of it. A bitmap of the entries' tokens in shared memory has a byte for each
// vector of eight; a warp looks at its vectors' bytes and takes out what is marked, which is
// rare. (Renormalised or not: the sum is over the others, and the entries are added.)
//
// A row is cut into pieces as in logprobs.cu. One warp of the block that is a row's last takes
// the teacher into its lanes' registers and finds the row's few logarithms; a duplicate token
// shows by its mark being there already, and only then the entries are compared with one
// another.
//
// Bound by memory: the loss of 1024 rows of 128256 bfloat16 takes 53 us (4.9 TB/s), of 4096
// rows 180 (5.8 TB/s).
#include "lp_finish.cuh"
#include "lp_stream.cuh"

namespace svl {
namespace {

// Turns that a block's bitmap of entries is for.
constexpr int32_t kSpan = kMostTurns;

struct DistillPlan {
    Cut cut;
    Split split;         // where rows are cut
};

// The teacher in its warp: entry lane + 32 q is the lane's q-th.
constexpr int kEach = SV_MAX_TOP / 32;
struct Teacher {
    int32_t id[kEach];   // -1 where there is none, or where its token came before
    float x[kEach];      // the student's logit
    float p[kEach];      // probability, before they are renormalised
    double mass;         // their sum
    float shift;         // what was taken off their logarithms
    int32_t distinct;
    int32_t status;
};

// The sum of a teacher's probabilities that are all there is: entropies of up to log 128 make its
// float32 logarithms' roundings 4.9 x 2^-24 of it, the exponentials' add 2 and the numbers' own 1; this
// is twice that.
constexpr double kRounding = 0x1p-20;

// Room for looking for entries of one token.
struct Entries {
    int32_t id[SV_MAX_TOP];
    float p[SV_MAX_TOP];
};

template <typename N>
__device__ __forceinline__ N warp_sum(N x)
{
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    return x;
}

// Takes the row's entries and their logits.
template <int DT>
__device__ __forceinline__ void read_teacher(Teacher& t, const DistillArgs& a, int32_t row,
                                             const uint8_t* x, int lane)
{
    int bad = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        const int j = lane + 32 * q;
        int32_t id = -1;
        float lp = -inf();
        if (j < a.k) {
            const int64_t at = static_cast<int64_t>(row) * a.k + j;
            id = a.ids[at];
            lp = a.logp[at];
        }
        const bool nonfinite = lp != lp || lp == inf();
        if (id < -1 || id >= a.r.V) bad |= SV_SEQ_BAD_TOKEN;
        if (nonfinite) bad |= SV_SEQ_NONFINITE;
        if (id < 0 || id >= a.r.V || nonfinite) {
            id = -1;
            lp = -inf();
        }
        t.id[q] = id;
        t.p[q] = lp;   // (its logarithm so far)
        t.x[q] = id >= 0 ? load_one<DT>(x, id) : 0.f;
    }
    t.status = __reduce_or_sync(0xFFFFFFFFu, bad);
}

// The entries' probabilities. `twice`: some token may have two entries.
__device__ __forceinline__ void make_teacher(Teacher& t, Entries& s, const DistillArgs& a, int lane,
                                             bool twice)
{
    // Renormalised probabilities are taken from the largest one, so that none overflows.
    t.shift = 0.f;
    if (!a.bucket) {
        float top = t.p[0];
#pragma unroll
        for (int q = 1; q < kEach; ++q) top = fmaxf(top, t.p[q]);
        top = warp_max(top);
        if (top != -inf()) t.shift = top;
    }
#pragma unroll
    for (int q = 0; q < kEach; ++q) t.p[q] = t.id[q] >= 0 ? expf(t.p[q] - t.shift) : 0.f;
    if (twice) {
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            s.id[lane + 32 * q] = t.id[q];
            s.p[lane + 32 * q] = t.p[q];
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            if (t.id[q] < 0) continue;
            float p = 0.f;
            bool first = true;
            for (int i = 0; i < a.k; ++i)
                if (s.id[i] == t.id[q]) {
                    first &= i >= lane + 32 * q;
                    p += s.p[i];
                }
            t.p[q] = first ? p : 0.f;
            if (!first) t.id[q] = -1;
        }
    }
    double mass = 0.0;
    int n = 0;
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        mass += t.p[q];
        n += t.id[q] >= 0;
    }
    t.mass = warp_sum(mass);
    t.distinct = __reduce_add_sync(0xFFFFFFFFu, n);
    // (Nothing to be renormalised; or more than float32 holds, as of logits given for probabilities.)
    if (a.bucket ? !(t.mass <= 3.40282347e38) : t.distinct > 0 && !(t.mass > 0.0))
        t.status |= SV_SEQ_NONFINITE;
}

// 1 / x to some 2^-40, for x in the range of floats.
__device__ __forceinline__ double inverse(double x)
{
    const double r = 1.0f / static_cast<float>(x);
    return r * (2.0 - x * r);
}

// Loss and gradient factors of a row, from the largest logit M_o and the sum S_o of
// 2^((x - M_o) c) over the tokens without entries (-inf and 0: none, or all of them are
// -inf). With M the largest of all, S the sum over all of 2^((x - M) c), q_e the entries'
// share of it and m the sum of their probabilities:
//   listed = 1 / S, scale = 2^((M_o - M) c) / S             renormalised
//   listed = max(m, 1) / S                                  bucket
//   scale  = (1 - P_o / q_o) 2^((M_o - M) c) / S = (m - q_e) / S_o     .. where m <= 1
// so that the others' gradient keeps its digits however small their share is.
__device__ __forceinline__ RowStats finish(const Teacher& t, const DistillArgs& a, int32_t row,
                                           float M_o, float S_o, int lane)
{
    RowStats st{};
    st.kind = kRowBad;
    const float c = a.r.c;
    float M = -inf();
#pragma unroll
    for (int q = 0; q < kEach; ++q)
        if (t.id[q] >= 0) M = fmax_nan(M, t.x[q]);
    M = fmax_nan(warp_max(M), M_o);
    if (!(fabsf(M) < inf()) || t.status != 0) {
        if (lane == 0) {
            if (a.loss != nullptr) a.loss[row] = nan();
            if (a.stats != nullptr) a.stats[row].kind = kRowBad;
            if (a.status != nullptr)
                a.status[row] = t.status | (fabsf(M) < inf() ? 0 : SV_SEQ_NONFINITE);
        }
        return st;
    }
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < kEach; ++q)
        if (t.id[q] >= 0) sum += ex2((t.x[q] - M) * c);
    const double S_e = warp_sum(sum);
    const float fall = S_o > 0.f ? ex2((M_o - M) * c) : 0.f;
    const double S = S_e + static_cast<double>(S_o) * fall;
    const double log_s = log_wide(static_cast<float>(S));
    const double over_mass = a.bucket ? 1.0 : inverse(t.mass);
    const double log_m = a.bucket ? 0.0 : log_wide(static_cast<float>(t.mass));
    double loss = 0.0;
#pragma unroll
    for (int q = 0; q < kEach; ++q)
        if (t.id[q] >= 0 && t.p[q] > 0.f)
            loss += t.p[q] * over_mass *
                    (log_wide(t.p[q]) - log_m - log_prob(t.x[q], M, c, log_s));
    loss = warp_sum(loss);
    const double over_S = inverse(S);
    float listed = static_cast<float>(over_S);
    float scale = listed * fall;
    if (a.bucket) {
        const double q_e = S_e * over_S;
        double P_o = t.distinct < a.r.V ? fmax(0.0, 1.0 - t.mass) : 0.0;
        // Tokens that a mask takes from student and teacher alike: what the entries leave them is the
        // rounding of their sum, and would be multiplied by the logarithm of a probability of 0.
        const bool none = !(S_o > 0.f) || fall == 0.f;
        if (none && P_o <= kRounding) P_o = 0.0;
        if (P_o > 0.0) {
            const float m = static_cast<float>(t.mass);
            const double log_P = m < 0.5f ? log1pf(-m) : logf(static_cast<float>(P_o));
            const double log_q = q_e < 0.5 ? static_cast<double>(log1pf(-static_cast<float>(q_e)))
                                           : log_prob(M_o, M, c, log_s) + log_wide(S_o);
            loss += P_o * (log_P - log_q);
        }
        listed = static_cast<float>((t.mass + P_o) * over_S);
        // (no other token, or all of probability 0: their gradient is 0)
        scale = !(S_o > 0.f)               ? 0.f
                : P_o > 0.0 && t.mass <= 1.0 ? static_cast<float>(t.mass - q_e) / S_o
                                             : listed * fall;
    }
    // (M_o where nothing is finite: any finite number)
    st = {S_o > 0.f ? M_o : 0.f,
          scale,
          0.f,
          M,
          listed,
          t.shift,
          static_cast<float>(over_mass),
          kRowGood};
    if (lane == 0) {
        if (a.loss != nullptr) a.loss[row] = static_cast<float>(loss);
        if (a.stats != nullptr) a.stats[row] = st;
        if (a.status != nullptr) a.status[row] = 0;
    }
    return st;
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

// A piece of a row to a block. SPLIT: of several. GRAD: a whole row, and its gradient after it.
template <int DT, bool SPLIT, bool GRAD>
__global__ void __launch_bounds__((GRAD ? kMostWarps : kLeastWarps) * 32, GRAD ? 2 : 8)
    distill_kernel(const __grid_constant__ DistillArgs a, const __grid_constant__ DistillPlan plan)
{
    constexpr int32_t kBits = kSpan * kTile * kPerVec<DT>;
    __shared__ uint32_t map[kBits / 32];
    __shared__ RowSum part[GRAD ? kMostWarps : kLeastWarps];
    __shared__ Entries entries;
    __shared__ uint32_t flag;
    // (GRAD: in shared memory, so that the loops' registers are not laid out for it)
    __shared__ Teacher teacher[GRAD ? 32 : 1];
    __shared__ RowStats done;
    const int32_t row = SPLIT ? row_of(plan.cut, blockIdx.x) : blockIdx.x, V = a.r.V;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const float c = a.r.c;
    if (!GRAD) sv::pdl_trigger();   // (the gradient's blocks, if there are to be any, may be launched)
    // Is there an entry, or a fault?
    int any = 0;
    for (int j = tid; j < a.k; j += blockDim.x) {
        const int64_t at = static_cast<int64_t>(row) * a.k + j;
        const float lp = a.logp[at];
        any |= a.ids[at] != -1 || lp != lp || lp == inf();
    }
    if (!__syncthreads_or(any)) {
        if (tid == 0 && (!SPLIT || part_of(plan.cut, blockIdx.x, row, 0).piece == 0)) {
            if (a.loss != nullptr) a.loss[row] = 0.f;
            if (a.stats != nullptr) a.stats[row].kind = kRowSkipped;
            if (a.status != nullptr) a.status[row] = 0;
        }
        if (GRAD) {
            const Vecs out = vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V);
            fill_tiles<DT>(out, warp, warps, tiles_of(out.n), V, 0.f);
        }
        return;
    }
    const Vecs in = vectors_of<DT>(row_begin(a.r.x, a.r.inner, row), V);
    const float step = kBehindSum / c, low = lowest_of<DT>(c);
    const int32_t tiles = tiles_of(in.n);
    const Part mine = SPLIT ? part_of(plan.cut, blockIdx.x, row, tiles) : Part{row, 0, 1, 0, tiles};
    const int32_t first = mine.first, end = mine.end;
    Running st;
    start(st);
    int32_t twice = 0;
    for (int32_t t0 = first; t0 < end; t0 += kSpan) {
        if (t0 > first) __syncthreads();
        for (int i = tid; i < kBits / 32; i += blockDim.x) map[i] = 0u;
        __syncthreads();
        const int64_t begin = static_cast<int64_t>(t0) * kTile * kPerVec<DT> - in.head;
        for (int j = tid; j < a.k; j += blockDim.x) {
            const int32_t id = a.ids[static_cast<int64_t>(row) * a.k + j];
            const int64_t at = id - begin;
            if (id < 0 || id >= V || at < 0 || at >= kBits) continue;
            const uint32_t was = atomicOr(&map[at >> 5], 1u << (at & 31));
            twice |= was >> (at & 31) & 1;
        }
        __syncthreads();
        const int32_t stop = min(t0 + kSpan, end);
        for (int32_t tile = t0 + warp; tile < stop; tile += warps) {
            uint4 v[kInFlight];
            ld_tile<DT>(v, in, tile * kTile, lane, V);
            uint32_t marks[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                marks[u] = marks_of<DT>(map, (tile - t0) * kTile + lane + u * 32);
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
    RowSum all = block_join(part, warp_join(st, twice, c), c);
    const bool cut = SPLIT && mine.pieces > 1;
    if (cut && !last_piece(plan.split, row - plan.cut.whole, mine, all, &flag)) return;
    if (!GRAD) {
        if (warp != 0) return;
        if (cut) all = join_pieces(plan.split, row - plan.cut.whole, mine.pieces, c, lane);
        Teacher t;
        read_teacher<DT>(t, a, row, in.a0 + in.head * kElem<DT>, lane);
        make_teacher(t, entries, a, lane, all.ahead != 0);
        finish(t, a, row, all.m, all.s, lane);
        return;
    }
    Teacher& t = teacher[lane];
    if (warp == 0) {
        read_teacher<DT>(t, a, row, in.a0 + in.head * kElem<DT>, lane);
        make_teacher(t, entries, a, lane, all.ahead != 0);
        const RowStats st = finish(t, a, row, all.m, all.s, lane);
        if (lane == 0) done = st;
    }
    __syncthreads();
    const Vecs out = vectors_of<DT>(row_begin(a.grad, a.r.inner, row), V);
    const float w = (a.weights == nullptr ? 1.f : a.weights[row]) * a.r.inv_t;
    if (done.kind != kRowGood) {
        fill_tiles<DT>(out, warp, warps, tiles_of(out.n), V, nan());
        return;
    }
    grad_tiles<DT, false>(in, out, warp, warps, tiles_of(out.n), V, done.M, c, w * done.scale, 0.f);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int q = 0; q < kEach; ++q)
        if (t.id[q] >= 0)
            store_one<DT>(out.a0 + out.head * kElem<DT>, t.id[q],
                          w * (done.listed * ex2((t.x[q] - done.listed_M) * c) - t.p[q] * done.inv));
}

// Loss and gradient by one block a row, in one launch, where rows are short or make one wave of
// blocks: what of them is still in L2 when the block comes to them again saves reads, and a
// launch is saved. In two launches the few rows of a call are cut finer. us, one and two, bfloat16:
//   rows              32        152       304       512       912        2000       8192
//   32000 (64 KB)     14 / 21   16 / 23   20 / 29   27 / 33   41 / 43    78 / 82    272 / 281
//   50257 (100 KB)    21 / 23   23 / 27   29 / 33   39 / 45   57 / 59    117 / 115
//   128256            29 / 23   35 / 35   49 / 53   76 / 80   123 / 123  262 / 248
// and float32 rows of 128256: 304 of them 84 / 87, 512 135 / 133. With 4, 8 and 16 warps a block,
// of 32000: 32 rows 23, 18 and 14; 456 rows 31, 27 and 31; 912 rows 41, 45 and 47. (The limits of 33, 50
// and 130 turns are those of the three vocabularies that were measured: 32, 50 and 126 turns. Where
// one way overtakes the other between them is not known.)
inline bool one_block(int64_t rows, int32_t tiles, bool grad)
{
    if (!grad) return false;
    return tiles <= 33 || (tiles <= 50 && rows * 4 <= kEnoughWarps) ||
           (tiles <= 130 && rows * 32 >= kEnoughWarps && rows * 8 <= kEnoughWarps);
}

template <int DT>
DistillPlan plan_of(const Rows& r, bool grad, int* warps)
{
    DistillPlan p{};
    const int32_t tiles = most_tiles(r.V, kPerVec<DT>);
    const bool one = one_block(r.rows, tiles, grad);
    p.cut = one ? Cut{r.rows, 1, tiles} : cut_of(r.rows, tiles, kLeastWarps, false);
    const int most = one ? warps_of(r.rows) : kLeastWarps;
    *warps = 1;
    while (*warps < most && *warps < p.cut.piece) *warps *= 2;
    return p;
}

template <int DT>
cudaError_t launch(const DistillArgs& a, void* workspace, bool* all_done, cudaStream_t s)
{
    int warps = 1;
    const bool grad = a.grad.base != nullptr;
    DistillPlan p = plan_of<DT>(a.r, grad, &warps);
    const bool cut = p.cut.pieces > 1;
    if (cut) p.split = split_of(workspace, a.r.rows - p.cut.whole, p.cut.pieces);
    const int32_t tiles = most_tiles(a.r.V, kPerVec<DT>);
    const bool one = one_block(a.r.rows, tiles, grad);
    const auto k = one             ? distill_kernel<DT, false, true>
                   : cut ? distill_kernel<DT, true, false>
                                  : distill_kernel<DT, false, false>;
    k<<<static_cast<unsigned>(blocks_of(p.cut, a.r.rows)), warps * 32, 0, s>>>(a, p);
    *all_done = one || !grad;
    return cudaGetLastError();
}

}  // namespace

size_t distill_workspace(const Rows& r, int dtype)
{
    int warps;
    const DistillPlan p = dtype == SV_F32 ? plan_of<SV_F32>(r, false, &warps)
                                          : plan_of<SV_BF16>(r, false, &warps);
    return p.cut.pieces > 1 ? split_bytes(r.rows - p.cut.whole, p.cut.pieces, 0) : 0;
}

cudaError_t launch_distill(const DistillArgs& a, int dtype, void* workspace, bool* all_done,
                           cudaStream_t s)
{
    return dtype == SV_F32    ? launch<SV_F32>(a, workspace, all_done, s)
           : dtype == SV_BF16 ? launch<SV_BF16>(a, workspace, all_done, s)
                              : launch<SV_F16>(a, workspace, all_done, s);
}

}  // namespace svl
