// lp_stream.cuh -- a row of logits through a block: its sums, and its gradient.
//
// A warp takes 128 vectors of 16 bytes at a time, four for each lane, and loads all of them
// before it uses the first. Vectors at a row's ends are looked at only where a warp's tile
// is not wholly inside; everywhere else a vector costs its load, a quarter of the loop's
// counting, and the arithmetic: five instructions an element for a sum with its entropy
// (pairs of float32 in one instruction where there is one), of the ten that there is time
// for at the memory's rate.
#pragma once

#include "lp_vec.cuh"

namespace svl {

constexpr int kInFlight = 4;                // vectors of a lane's turn
constexpr int kTile = 32 * kInFlight;       // vectors of a warp's turn

// The largest |x c| that is taken off in one instruction with the product (t = x c - o).
// Rows of logits further from 0 subtract first, since o would be rounded to a multiple of
// something that matters.
constexpr float kNear = 1048576.f;

// A thread's sums of 2^t and 2^t t, t = x c - o, where o is (about) the largest x c seen, behind it
// by so many bits at most: it moves hardly ever. A sum of 2^t alone takes no harm from that. In one
// of 2^t t a largest element whose t is d weighs d times what it does with o at the element itself,
// and so does every rounding after it, though nearly all of that is taken off again at the end. Log
// probabilities of rows of 128256 at temperature 0.7: 16 bits leave the entropies 3.5e-7 off in norm and
// 8.6e-6 at most, 8 leave 0.85e-7 and 1.3e-6, 4 and fewer 0.71e-7 and 1.2e-6; 4096 rows take 167, 168
// and 171 us, 256 x 9 ragged ones with 20 alternatives 80, 81 and 83.
constexpr float kBehindSum = 16.f, kBehindEntropy = 8.f;
struct Running {
    float m;            // largest logit (NaN if there is one)
    float r;            // the logit that o stands for; -inf: none yet
    float limit;        // a logit above this moves it
    float o;            // r c rounded
    bool near;          // or, far from 0: t = (x - r) c
    uint64_t s, e;      // two sums each
};

__device__ __forceinline__ void start(Running& st)
{
    st.m = st.r = st.limit = -inf();
    st.o = 0.f;
    st.near = false;
    st.s = st.e = pack2(0.f, 0.f);
}

// What t is relative to, exactly.
__device__ __forceinline__ double reference(const Running& st, float c)
{
    return st.near ? static_cast<double>(st.o) : static_cast<double>(st.r) * c;
}

// Sums against another reference, d = old - new further down (or, on the last step, up by
// no more than kBehindSum).
__device__ __forceinline__ void rebase(float& s, float& e, float d)
{
    d = fmaxf(d, -1000.f);
    const float f = ex2(d);
    e = fmaf(s, d, e) * f;
    s *= f;
}

static __device__ __noinline__ Running moved(Running st, float to, float c, float step, float low)
{
    const Running old = st;
    st.r = to;
    st.o = to * c;
    st.limit = to + step;
    st.near = fabsf(st.o) < kNear && (to - low) * c > 256.f;
    if (old.r != -inf()) {
        const float d = old.near && st.near
                            ? old.o - st.o
                            : static_cast<float>(reference(old, c) - reference(st, c));
        float s0, s1, e0, e1;
        unpack2(st.s, s0, s1);
        unpack2(st.e, e0, e1);
        rebase(s0, e0, d);
        rebase(s1, e1, d);
        st.s = pack2(s0, s1);
        st.e = pack2(e0, e1);
    }
    return st;
}

// A logit below this has no share in a sum whose reference is near 0 (and 256 / c above it,
// which float16's end may not be), and t is finite for it: masked logits, -inf among them, are
// raised to it, or 2^t t would be 0 times infinity.
template <int DT>
__device__ __forceinline__ float lowest_of(float c)
{
    const float l = -2.f * kNear / c;
    const float end = DT == SV_F16 ? -65504.f : -3.3895314e38f;
    const float x = fmaxf(l, end);
    return DT == SV_F32 ? x : DT == SV_BF16 ? __bfloat162float(__float2bfloat16_rn(x))
                                            : __half2float(__float2half_rn(x));
}
template <int DT>
__device__ __forceinline__ uint32_t pair_of(float x)
{
    if (DT == SV_F32) return __float_as_uint(x);
    const uint32_t h = DT == SV_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                                     : __half_as_ushort(__float2half_rn(x));
    return h | h << 16;
}
// (not the maximum that hands NaN on: rows with NaN are told by their maximum)
template <int DT>
__device__ __forceinline__ uint32_t raised(uint32_t w, uint32_t low)
{
    uint32_t r;
    if (DT == SV_F32)
        asm("max.f32 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
    else if (DT == SV_BF16)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
    else
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
    return r;
}

template <int DT, bool ENTROPY>
__device__ __forceinline__ void add_tile(Running& st, const uint4 (&v)[kInFlight], float c,
                                         uint32_t low)
{
    const uint64_t o2 = pack2(-st.o, -st.o), c2 = pack2(c, c);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
        uint4 w = v[u];
        if (ENTROPY)
            w = make_uint4(raised<DT>(w.x, low), raised<DT>(w.y, low), raised<DT>(w.z, low),
                           raised<DT>(w.w, low));
        uint64_t p[kPerVec<DT> / 2];
        widen<DT>(w, p);
#pragma unroll
        for (int i = 0; i < kPerVec<DT> / 2; ++i) {
            const uint64_t t = fma2(p[i], c2, o2);
            float a, b;
            unpack2(t, a, b);
            const uint64_t e = pack2(ex2(a), ex2(b));
            st.s = add2(st.s, e);
            if (ENTROPY) st.e = fma2(e, t, st.e);
        }
    }
}

// The same for a reference far from 0.
template <int DT>
__device__ __noinline__ void add_far(Running* st, uint4 v, float c)
{
    const uint64_t r2 = pack2(-st->r, -st->r), c2 = pack2(c, c);
    uint64_t p[kPerVec<DT> / 2];
    widen<DT>(v, p);
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) {
        float a, b;
        unpack2(mul2(add2(p[i], r2), c2), a, b);
        a = fmaxf(a, -1000.f);
        b = fmaxf(b, -1000.f);
        const uint64_t e = pack2(ex2(a), ex2(b));
        st->s = add2(st->s, e);
        st->e = fma2(e, pack2(a, b), st->e);
    }
}

// One turn's vectors, whose largest element is `top`, into a thread's sums.
template <int DT, bool ENTROPY>
__device__ __forceinline__ void take(Running& st, const uint4 (&v)[kInFlight], float top, float c,
                                     float step, float low)
{
    st.m = fmax_nan(st.m, top);
    if (top > st.limit) st = moved(st, top, c, step, low);
    if (st.near) {
        add_tile<DT, ENTROPY>(st, v, c, pair_of<DT>(low));
    } else if (st.r != -inf()) {  // (-inf: nothing but that so far)
        Running copy = st;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) add_far<DT>(&copy, v[u], c);
        st = copy;
    }
}

// A warp's turn lies wholly inside a row.
__device__ __forceinline__ bool whole(const Vecs& r, int32_t base)
{
    return base >= r.full && base + kTile <= r.full_end;
}

// Vectors j, j + 32, .. of a row; -inf where it has none.
template <int DT>
__device__ __forceinline__ void ld_tile(uint4 (&v)[kInFlight], const Vecs& in, int32_t base, int lane,
                                        int32_t V)
{
    if (whole(in, base)) {
        const uint8_t* p = in.a0 + static_cast<int64_t>(base + lane) * 16;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) v[u] = ld_stream(p + u * 512);
    } else {
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) v[u] = ld_vec<DT>(in, base + lane + u * 32, V);
    }
}

// What is known of (a part of) a row: sums of 2^t and 2^t t with t = (x - m) c.
struct __align__(16) RowSum {
    float m;            // largest logit (NaN, +inf: a bad row; -inf: nothing else)
    float s, e;
    int32_t ahead;      // tokens ahead of the given one
};

__device__ __forceinline__ RowSum join(RowSum a, RowSum b, float c)
{
    RowSum r;
    r.m = fmax_nan(a.m, b.m);
    if (a.s > 0.f) rebase(a.s, a.e, (a.m - r.m) * c);
    if (b.s > 0.f) rebase(b.s, b.e, (b.m - r.m) * c);
    r.s = a.s + b.s;
    r.e = a.e + b.e;
    r.ahead = a.ahead + b.ahead;
    return r;
}

// The sums of a warp's lanes, in all of them.
__device__ __forceinline__ RowSum lanes_join(RowSum r, float c)
{
    const float m = warp_max(r.m);
    if (r.s > 0.f) rebase(r.s, r.e, (r.m - m) * c);
    r.m = m;
    for (int off = 16; off > 0; off >>= 1) {
        r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, off);
        r.e += __shfl_xor_sync(0xFFFFFFFFu, r.e, off);
    }
    r.ahead = __reduce_add_sync(0xFFFFFFFFu, r.ahead);
    return r;
}

// The same of their running sums.
__device__ __forceinline__ RowSum warp_join(const Running& st, int32_t ahead, float c)
{
    RowSum r;
    r.m = warp_max(st.m);
    float s0, s1, e0, e1;
    unpack2(st.s, s0, s1);
    unpack2(st.e, e0, e1);
    r.s = s0 + s1;
    r.e = e0 + e1;
    if (r.s > 0.f)  // (o - m c, rounded once)
        rebase(r.s, r.e, st.near ? fmaf(-r.m, c, st.o) : (st.r - r.m) * c);
    for (int off = 16; off > 0; off >>= 1) {
        r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, off);
        r.e += __shfl_xor_sync(0xFFFFFFFFu, r.e, off);
    }
    r.ahead = __reduce_add_sync(0xFFFFFFFFu, ahead);
    return r;
}

// e (A + B t) with t = (x - M) c and e = 2^t, for the vectors of a gradient's row that are in
// the warps' turns first_tile, first_tile + step, .. before end_tile.
template <int DT, bool LINEAR>
__device__ __forceinline__ void grad_tiles(const Vecs& in, const Vecs& out, int32_t first_tile,
                                           int32_t step, int32_t end_tile, int32_t V, float M,
                                           float c, float A, float B)
{
    constexpr int P = kPerVec<DT> / 2;
    const int lane = threadIdx.x & 31;
    const Shift sh = shift_of<DT>(in, out);
    const uint64_t m2 = pack2(-M, -M), c2 = pack2(c, c), A2 = pack2(A, A), B2 = pack2(B, B);
    for (int32_t tile = first_tile; tile < end_tile; tile += step) {
        const int32_t base = tile * kTile;
        const bool inside = whole(out, base);
        uint4 v[kInFlight];
        if (sh.shift == 0) {
            ld_tile<DT>(v, in, base, lane, V);
        } else {
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int32_t i = base + lane + u * 32 + sh.step;
                // (vectors around the row's: -inf, nothing is loaded)
                const uint4 a = ld_vec<DT>(in, i < 0 ? in.n : i, V);
                const uint4 b = ld_vec<DT>(in, i + 1, V);
                v[u] = shifted(a, b, sh.shift * kElem<DT>);
            }
        }
        uint8_t* g = out.a0 + static_cast<int64_t>(base + lane) * 16;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            uint64_t p[P];
            widen<DT>(v[u], p);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                uint64_t t = mul2(add2(p[i], m2), c2);
                float t0, t1;
                unpack2(t, t0, t1);
                if (LINEAR) {
                    // (masked logits: 0 times a number and not times -inf)
                    t0 = fmaxf(t0, -1000.f);
                    t1 = fmaxf(t1, -1000.f);
                    t = pack2(t0, t1);
                }
                const uint64_t e = pack2(ex2(t0), ex2(t1));
                p[i] = mul2(e, LINEAR ? fma2(B2, t, A2) : A2);
            }
            const uint4 w = narrow<DT>(p);
            if (inside)
                st_stream(g + u * 512, w);
            else
                st_vec<DT>(out, base + lane + u * 32, V, w);
        }
    }
}

// One value throughout the same vectors.
template <int DT>
__device__ __forceinline__ void fill_tiles(const Vecs& out, int32_t first_tile, int32_t step,
                                           int32_t end_tile, int32_t V, float value)
{
    const uint64_t f = pack2(value, value);
    uint64_t p[kPerVec<DT> / 2];
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) p[i] = f;
    const uint4 v = narrow<DT>(p);
    for (int32_t tile = first_tile; tile < end_tile; tile += step)
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            st_vec<DT>(out, tile * kTile + (threadIdx.x & 31) + u * 32, V, v);
}

__host__ __device__ __forceinline__ int32_t tiles_of(int64_t vectors)
{
    return static_cast<int32_t>((vectors + kTile - 1) / kTile);
}

// Most turns of a row of V elements, which may begin anywhere. (V up to 2^31 - 1, and elements in
// front of the row: sums of them need 64 bits.)
__host__ __device__ __forceinline__ int32_t most_tiles(int32_t V, int per_vec)
{
    return tiles_of((static_cast<int64_t>(V) + per_vec - 1) / per_vec + 1);
}

// Rows in pieces, a block each. What the pieces leave for one another lies in the workspace: a
// counter a row, in a place of their own that other calls' workspaces have too, since the
// counters are 0 between calls; then the pieces' sums; then the groups' maxima.
constexpr int64_t kMaxSplitRows = 65536;   // (no more than 4864 are cut)
constexpr int32_t kMostTurns = 32;         // of a bitmap of entries
constexpr int64_t kEnoughWarps = 4864;     // 32 an SM

struct Split {
    uint32_t* counters;
    RowSum* sums;
    float* maxima;
};

// Warps of a block that has much to do after its sums: 4, or up to 16 where that makes no more of
// them than run at a time, 32 an SM.
constexpr int kLeastWarps = 4, kMostWarps = 16;
inline int warps_of(int64_t rows)
{
    int warps = kMostWarps;
    while (warps > kLeastWarps && warps * rows > kEnoughWarps) warps /= 2;
    return warps;
}

// Rows [0, whole) are a block each; the others are cut into `pieces` of `piece` turns.
struct Cut {
    int32_t whole, pieces, piece;
};
inline int64_t blocks_of(const Cut& c, int64_t rows) { return c.whole + (rows - c.whole) * c.pieces; }

// How rows of so many turns are cut. All of them, if they are few: into as many pieces as make
// one wave of blocks, with two turns a warp at least: more blocks than run at a time end in a wave that
// is not full, and a block's beginning and end cost as much as three turns a warp. For 1024 rows of
// 128256 (bfloat16, without alternatives): one piece 52 us, two 62, four 56, eight 58; 544 rows:
// 41, 35, 38, 38; 40 rows: 35, 23, 17, 15. If there are more long rows than run at a time, those of
// a last wave that is at most half full: losses of 1400, 2048 and 4096 rows, all whole 88, 99 and
// 182, all in two 78, 107 and 191, so 72, 99 and 179; but of 4096 rows of 64 KB 68, and so 70.
// `ragged` (with alternatives): somewhat more long rows than run at a time are all cut in two, since
// some may have nothing to do: 2304 rows with 20 alternatives, half of the rows empty, one piece
// 96, two 86 (blocks of two warps 106); 1280 full rows 99 and 87; but 2304 full ones 125 and 135. (Rows
// of calls without tokens are never empty, and are cut all the same.)
inline Cut cut_of(int64_t rows, int32_t tiles, int32_t warps, bool ragged)
{
    const Cut none{static_cast<int32_t>(rows), 1, tiles};
    if (rows == 0) return none;
    const int64_t blocks = kEnoughWarps / warps;
    int64_t whole = 0, n = 1;
    if (rows <= blocks) {
        n = blocks / rows;
    } else if (tiles < 64) {
        return none;
    } else if (ragged) {
        if (rows < 4 * blocks) n = 2;
    } else {
        whole = rows / blocks * blocks;
        n = rows > whole ? blocks / (rows - whole) : 1;
    }
    if (n > tiles / (2 * warps)) n = tiles / (2 * warps);
    if (n <= 1) return none;
    // (evenly, in whole turns of all warps)
    const int64_t piece = ((tiles + n - 1) / n + warps - 1) / warps * warps;
    const Cut cut{static_cast<int32_t>(whole), static_cast<int32_t>((tiles + piece - 1) / piece),
                  static_cast<int32_t>(piece)};
    // (a grid ends at 2^31 - 1 blocks, and rows may be as many)
    return blocks_of(cut, rows) < (int64_t(1) << 31) ? cut : none;
}

// A gradient's rows: a warp has up to four turns, in blocks of one to eight warps: short rows leave
// few threads idle, long ones are cut where a block's start no longer shows.
constexpr int kGradWarps = 8;
struct GradPlan {
    int32_t pieces;          // of a row
    int32_t piece;           // warps' turns in a piece
};
inline GradPlan grad_plan_of(int32_t rows, int32_t tiles, int* warps)
{
    *warps = 1;
    while (*warps < kGradWarps && *warps < tiles) *warps *= 2;
    int64_t piece = *warps * 4, pieces = (tiles + piece - 1) / piece;
    while (pieces * rows >= (int64_t(1) << 31)) {
        piece *= 2;
        pieces = (tiles + piece - 1) / piece;
    }
    return {static_cast<int32_t>(pieces), static_cast<int32_t>(piece)};
}

// A block's part of a row.
struct Part {
    int32_t row, piece, pieces;
    int32_t first, end;     // turns
};
__device__ __forceinline__ int32_t row_of(const Cut& c, int32_t block)
{
    return block < c.whole ? block : c.whole + (block - c.whole) / c.pieces;
}
__device__ __forceinline__ Part part_of(const Cut& c, int32_t block, int32_t row, int32_t tiles)
{
    if (block < c.whole) return {row, 0, 1, 0, tiles};
    const int32_t piece = block - c.whole - (row - c.whole) * c.pieces, first = piece * c.piece;
    return {row, piece, c.pieces, first, min(first + c.piece, tiles)};
}

// (rows that are cut, here and further down: counted from the first one)
inline size_t split_bytes(int64_t rows, int64_t pieces, int64_t groups)
{
    return kMaxSplitRows * 4 + static_cast<size_t>(rows) * pieces * sizeof(RowSum) +
           static_cast<size_t>(rows) * groups * 4;
}

inline Split split_of(void* workspace, int64_t rows, int64_t pieces)
{
    Split s;
    s.counters = static_cast<uint32_t*>(workspace);
    s.sums = reinterpret_cast<RowSum*>(s.counters + kMaxSplitRows);
    s.maxima = reinterpret_cast<float*>(s.sums + rows * pieces);
    return s;
}

// The sums of a block's warps, in the first warp's lanes (part: a place for each warp; `mine`:
// in all lanes). Ends after a barrier.
__device__ __forceinline__ RowSum block_join(RowSum* part, const RowSum& mine, float c)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = mine;
    __syncthreads();
    RowSum r{-inf(), 0.f, 0.f, 0};
    if (threadIdx.x < 32) {
        if (lane < warps) r = part[lane];
        r = lanes_join(r, c);
    }
    return r;
}

// Leaves a piece's sums (those of thread 0) and says whether all of the row's are there now;
// everything that the block's threads wrote before is then visible to the block that is told so,
// past the first-level cache.
__device__ __forceinline__ bool last_piece(const Split& s, int32_t row, const Part& p,
                                           const RowSum& mine, uint32_t* shared)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __stcg(reinterpret_cast<float4*>(s.sums + static_cast<int64_t>(row) * p.pieces + p.piece),
               make_float4(mine.m, mine.s, mine.e, __int_as_float(mine.ahead)));
        // (releases what the barrier has shown this thread of the others' writes too)
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                     : "=r"(before)
                     : "l"(s.counters + row), "r"(static_cast<uint32_t>(p.pieces - 1))
                     : "memory");
        *shared = before == static_cast<uint32_t>(p.pieces - 1);
    }
    __syncthreads();
    return *shared != 0;
}

// A row's sums from its pieces', in all threads; by each warp for itself, in one order.
__device__ __forceinline__ RowSum join_pieces(const Split& s, int32_t row, int32_t pieces, float c,
                                              int lane)
{
    RowSum r{-inf(), 0.f, 0.f, 0};
    const float4* p = reinterpret_cast<const float4*>(s.sums + static_cast<int64_t>(row) * pieces);
    for (int32_t i = lane; i < pieces; i += 32) {
        const float4 f = __ldcg(p + i);
        r = join(r, {f.x, f.y, f.z, __float_as_int(f.w)}, c);
    }
    return lanes_join(r, c);
}

}  // namespace svl
