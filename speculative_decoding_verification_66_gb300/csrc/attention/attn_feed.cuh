// attn_feed.cuh -- what the attention kernels that work by 128-key tiles share:
// the plan of a block's segments, the loads of keys and values into a ring of
// shared-memory stages, e4m3, rows computed again, and the joining of items that
// several blocks worked on.
#pragma once

#include <atomic>
#include <climits>
#include <type_traits>

#include "attn_internal.h"
#include "attn_plan.cuh"
#include "tensor_core.cuh"

namespace sva {
namespace {

// The outputs are rescaled when a weight would pass 2^slack(); the largest weight
// is then 2^rise(). float16 weights stay below 65504 (e4m3 caches: also after a
// tile's exponent, see kLift) and start well above 1: what is lost below their
// least step 2^-24, for each of many keys in the same direction, is 2^-32 of the
// largest weight (e4m3: 2^-27; with a start at 1 and tiles 2^6 below the
// reference 131072 keys of 2^-19.5 would vanish, a seventh of the sum). bfloat16
// has float32's range; slack 30 leaves sums room for values up to 2^90.
template <class T, bool E4M3>
__device__ __forceinline__ float slack()
{
    return E4M3 ? 8.f : std::is_same<T, F16>::value ? 14.f : 30.f;
}
template <class T, bool E4M3>
__device__ __forceinline__ float rise()
{
    return E4M3 ? 4.f : std::is_same<T, F16>::value ? 7.f : 0.f;
}
// e4m3: the weights carry the power of two between their tile's values and the
// outputs' reference, which follows the tiles when they are more than kLift above
// or kSink below.
constexpr int kLift = 7, kSink = 2;
// Keys or values of one tile may be this many powers of two apart (see code_factor).
constexpr int kSpread = 22;
// The values of a segment's tiles may be this many powers of two apart: outputs that
// follow them stay below 2^127 (values 2^16, weights 2^15, 2^30 keys), and moved() is
// exact. Beyond, the segment's rows are computed again.
constexpr int kFar = 60;
// A row's scores are below 2^38 before they are multiplied by its query's factor and
// by the key's exponent, in either order: exponent bytes above kLarge (2^60) or a
// factor above 2^67 might overflow on the way where the product does not. All rows
// are computed again.
constexpr uint32_t kLarge = 127 + 60;

constexpr int kMaxBlocks = 160;  // shares in the workspace; grids are no larger
constexpr size_t kMaxSmem = 232448;
constexpr int kNoted = 4;        // noted positions a segment can hold
constexpr int kItems = 16;       // segments whose plans and notes are kept at one time

// A segment as the warps need it. Positions count from the segment's first
// tile; tiles are numbered from it.
struct Plan {
    int32_t n;                         // tiles; 0: no more segments
    int32_t b, h, q0, row0, rows;
    int32_t tile0;                     // the first tile's number in the sequence
    int32_t cached;                    // row r stands at position cached + r / G
    int32_t low;                       // .. and sees positions from low + r / G on
    int32_t lo0, hi0, lo1, hi1;        // split in two slots of 128 rows: their tiles
    int32_t any_lo, any_hi;            // positions that some row sees
    int32_t all_lo, all_hi;            // positions that every row sees
    int32_t inner_lo, inner_hi;        // tiles wholly in `all`; the others have hidden values
    int32_t begins, whole;             // the item begins here; is all here
};

struct Tiles {
    Attn a;
    float* part;   // [blocks][2][rows][part_cols]: unnormalised O, then m and l
    Share* shares; // [blocks]
    int32_t* failed;  // [blocks]: a bounded wait ran out in this block
    int32_t part_rows;
    int32_t swizzled;  // e4m3 rows of 128 or 64 bytes lie swizzled (few rows)
};

// A tile of 16-bit elements in shared memory: panels of 64 elements of every row,
// rows of 128 bytes, swizzled.
constexpr int kPanel = kTile * 128;

constexpr size_t kShareBytes = (sizeof(Share) * kMaxBlocks + 255) / 256 * 256;
constexpr size_t kFailedBytes = (sizeof(int32_t) * kMaxBlocks + 255) / 256 * 256;

// Which 16 bytes of a row of codes hold chunk `ch`: swizzled as bulk tensor copies
// do it, rows of 128 bytes by the row, of 64 bytes by every second row.
template <int DP>
__device__ __forceinline__ int few_swizzle(int row, int ch, int swizzled)
{
    return DP <= 128 && swizzled ? (DP == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3)) : ch;
}

// Where the tiles of a segment lie in the ring: the order in which the products
// use them: K0 V0 K1 V1 ..; ALT: K0 K1 V0 K2 V1 .., where the next tile's scores
// come before a tile's values.
template <bool ALT>
__device__ __forceinline__ int ring_v(int k, int n)
{
    return ALT && k < n - 1 ? 2 * k + 2 : 2 * k + 1;
}
// From a tile's keys, and its values, to the next tile's.
template <bool ALT>
__device__ __forceinline__ int ring_k_step(int k)
{
    return ALT && k == 0 ? 1 : 2;
}
template <bool ALT>
__device__ __forceinline__ int ring_v_step(int k, int n)
{
    return ALT && k == n - 2 ? 1 : 2;
}

// A place in a ring of S stages, and the round it is in.
template <int S>
struct Place {
    int stage = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void advance(int n)
    {
        stage += n;
        while (stage >= S) {
            stage -= S;
            ++round;
        }
    }
};

// Positions of a segment are far below 2^30; those outside need not be told apart.
__device__ __forceinline__ int clamp32(int64_t v)
{
    return static_cast<int>(max(min(v, int64_t(INT_MAX / 2)), int64_t(INT_MIN / 2)));
}

template <bool SPLIT>
__device__ __forceinline__ Plan plan_of(const Attn& a, const Segment& g)
{
    Plan p;
    const int64_t origin = static_cast<int64_t>(g.t.lo) << kTileShift;
    const int r1 = g.row0 + g.rows - 1;
    const int64_t p0 = g.cached + g.row0 / a.G, p1 = g.cached + r1 / a.G;
    p.n = g.t.hi - g.t.lo;
    p.b = g.b;
    p.h = g.h;
    p.q0 = g.q0;
    p.row0 = g.row0;
    p.rows = g.rows;
    p.tile0 = g.t.lo;
    p.cached = clamp32(g.cached - origin);
    p.low = a.window > 0 ? clamp32(g.cached - a.window + 1 - origin) : INT_MIN / 2;
    p.any_lo = clamp32(first_key(a, p0) - origin);
    p.any_hi = clamp32(p1 - origin);
    p.all_lo = clamp32(first_key(a, p1) - origin);
    p.all_hi = clamp32(p0 - origin);
    p.inner_lo = (p.all_lo + kTile - 1) >> kTileShift;
    p.inner_hi = ((p.all_hi + 1) >> kTileShift) - 1;
    p.begins = g.t.lo == g.item.lo;
    p.whole = p.begins && g.t.hi == g.item.hi;
    p.lo0 = p.lo1 = 0;
    p.hi0 = p.hi1 = p.n;
    if (SPLIT) {
        const Range t0 = row_tiles(a, g.cached, g.row0, g.row0 + min(g.rows, 128));
        p.lo0 = max(t0.lo - g.t.lo, 0);
        p.hi0 = min(t0.hi - g.t.lo, p.n);
        p.hi1 = 0;
        if (g.rows > 128) {
            const Range t1 = row_tiles(a, g.cached, g.row0 + 128, g.row0 + g.rows);
            p.lo1 = max(t1.lo - g.t.lo, 0);
            p.hi1 = min(t1.hi - g.t.lo, p.n);
        }
    }
    return p;
}

// ---------------------------------------------------------------------------
// Expanding e4m3 to float16, relative to the largest exponent `top` of a tile:
// code 2^(kUp + e - top), the conversion and one multiplication for two values. Codes
// have three mantissa bits, a least step of 2^-9 and are at most 448, which kUp = 7
// brings to 57344: this is exact for top - e <= kSpread = 22 (2^-24, float16's least).
// Rows of tiles whose vectors lie further apart are computed again, key by key, which
// takes a hundred times as long and more; so the range counts.
// ---------------------------------------------------------------------------
constexpr int kUp = 7;
constexpr float kDown = 1.f / (1 << kUp);
__device__ __forceinline__ uint32_t both(uint32_t h) { return h | (h << 16); }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Four codes to two words of float16.
__device__ __forceinline__ uint2 spread(uint32_t w)
{
    uint2 r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(w));
    return r;
}
// The factor of a vector's codes, in both halves.
__device__ __forceinline__ uint32_t code_factor(uint32_t e, uint32_t top)
{
    if (e == 255u) return both(0x7FFFu);
    const int d = static_cast<int>(top) - static_cast<int>(e);
    return both(d <= 14 + kUp   ? static_cast<uint32_t>(15 + kUp - d) << 10
                : d <= 24 + kUp ? 1u << (24 + kUp - d)
                                : 0u);
}
// 16 codes times a factor, as sixteen float16 values.
__device__ __forceinline__ void expand(uint4 codes, uint32_t f, uint32_t (&o)[8])
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint2 s = spread(w[i]);
        o[2 * i] = mul2(s.x, f);
        o[2 * i + 1] = mul2(s.y, f);
    }
}
// Exponent bytes up to kLeast stand for vectors of zeros, nearly always (10), and for
// vectors of next to nothing (up to 448 2^-87). Zeros must not move a tile's or the
// outputs' exponent, so these vectors are left out there. Somebody looks at their
// codes, and where one is not zero all rows are computed again: with few rows the
// loads, from memory, behind the workers' backs (131k keys 231 us; anywhere in the
// workers' loop 240 and more, against 229 without); in the tile kernel, whose loading
// warps have no registers for it (256 x 9 tokens 753 us), the helpers, whom a factor of
// minus zero tells which rows (660, against 655 without).
constexpr uint32_t kLeast = 40, kUnless = 0x8000u;
__device__ __forceinline__ bool not_zeros(uint4 codes)
{
    return ((codes.x | codes.y | codes.z | codes.w) & 0x7F7F7F7Fu) != 0;
}
// Whether the outputs' reference exponent (0: none yet) has to move to a tile's,
// and the power of two that the outputs are then multiplied by. Tiles that have no
// values above kLeast (0: none visible) do not count.
__device__ __forceinline__ bool moves(int ref, int top)
{
    return top > static_cast<int>(kLeast) && (ref == 0 || top - ref > kLift || ref - top > kSink);
}
__device__ __forceinline__ float moved(int ref, int top)
{
    return ref == 0 ? 1.f : exp_value(static_cast<uint32_t>(max(min(127 + ref - top, 227), 27)));
}

// The exponent (biased) that a bfloat16 query row is scaled by, from the bits of its
// largest element. A row with an infinity or a NaN has nothing to lose: its size is 1.
__device__ __forceinline__ int row_exponent(uint32_t top)
{
    const int e = max(static_cast<int>(top >> 23), 15);
    return e == 255 ? 127 + 14 : e;
}
// The query's part of the factor of a row's scores: the scale and its power of two.
__device__ __forceinline__ float row_factor(float c, int* noted)
{
    if (c > __uint_as_float((127u + 67u) << 23)) atomicAdd(noted, kNoted + 1);  // (see kLarge)
    return c;
}
// The factor of a row's scores: the above and the keys' power of two. Where these
// multiply to nothing (a row of zeros, keys of zeros) a hidden score's -inf times zero
// would be NaN. Scores are below 2^38 before this factor (few rows: times a key's
// exponent, 2^91), so the least normal number in the place of a smaller one moves none
// by 2^-88 (2^-35).
__device__ __forceinline__ float score_factor(float c)
{
    return fmaxf(c, __uint_as_float(0x00800000u));
}

// A weight is 2^(s c - m), by one rounding, with m the rounded product of the largest
// score: where that is so large that its own rounding counts, the largest weight would
// be anything up to infinity. Such rows are computed again, where scores are rounded
// before they are compared. (Below 2^22 the weights are off by the square root of 2 at
// most, which their types have room for.)
// Asked whenever m moves. Where it is infinite the row is NaN either way.
__device__ __forceinline__ bool too_far(float m)
{
    return fabsf(m) > 4194304.f && m < __uint_as_float(0x7F800000u);
}

// Notes that all rows of a segment have to be computed again. (A plain store: the
// number only has to stay above kNoted.)
__device__ __forceinline__ void note_all(int* noted)
{
    *reinterpret_cast<volatile int*>(noted) = kNoted + 1;
}

__device__ __forceinline__ bool any_special(uint4 w, uint32_t exponent)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    bool s = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s |= (u[i] & exponent) == exponent || ((u[i] >> 16) & exponent) == exponent;
    return s;
}
__device__ __forceinline__ uint32_t exponent_mask(Bf16) { return 0x7F80u; }
__device__ __forceinline__ uint32_t exponent_mask(F16) { return 0x7C00u; }

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Byte offset of 16-byte chunk `chunk` of a row in a tile (see kPanel).
__device__ __forceinline__ uint32_t tile_chunk(int row, int chunk)
{
    return (chunk >> 3) * kPanel + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// Where this block starts, into ctl.start. True if some sequence's lengths are
// bad. The sequences' units are added up THREADS at a time; with no more
// sequences than threads the one pass finds the start too.
template <int R, int THREADS, class Ctl>
__device__ bool find_start(const Attn& a, Ctl& ctl)
{
    constexpr int kWarps = THREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t U = 0, u = 0, scan = 0, chunk = 0;
    bool bad = false;
    // Units of sequence base + tid, their sum up to it, and the sum of all of the
    // pass.
    auto pass = [&](int64_t base) {
        const int64_t b = base + tid;
        u = 0;
        if (b < a.c.B) {
            const Seq q = seq_of(a.c, static_cast<int>(b), a.tokens, a.max_chunk);
            bad |= q.bad != 0;
            u = head_units<R>(a, q) * a.c.Hkv;
        }
        scan = u;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, scan, d);
            if (lane >= d) scan += o;
        }
        __syncthreads();
        if (lane == 31) ctl.sums[warp] = scan;
        __syncthreads();
        chunk = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) scan += ctl.sums[w];
            chunk += ctl.sums[w];
        }
    };
    for (int64_t base = 0; base < a.c.B; base += THREADS) {
        pass(base);
        U += chunk;
    }
    const int64_t u0 = share_begin(U, blockIdx.x, gridDim.x);
    const int64_t u1 = share_begin(U, blockIdx.x + 1, gridDim.x);
    if (tid == 0) ctl.start = Start{u0, u1, U, 0, 0};
    __syncthreads();
    if (u0 < u1) {
        int64_t before = 0;
        for (int64_t base = 0; base < a.c.B && before <= u0; base += THREADS) {
            if (a.c.B > THREADS) pass(base);
            const int64_t begin = before + scan - u;
            if (u0 >= begin && u0 < begin + u) {
                ctl.start.off = u0 - begin;
                ctl.start.b = static_cast<int32_t>(base + tid);
            }
            before += chunk;
        }
    }
    return __syncthreads_or(bad) != 0;
}

// Sequences whose lengths are bad: their rows become NaN, but for those that belong to
// a good one; block c of n takes sequences c, c + n, .. Where the starts are out of
// order, so that rows of two sequences may be the same, the call's good rows are
// computed here, row by row, and the blocks are left without work. (Not inlined, and
// nothing of it in the ordinary path: sequences that were checked one by one in the
// plan cost 256 x 9 e4m3 tokens 120 us of 660.)
template <class T, bool E4M3, class Ctl>
__device__ __noinline__ void refuse_sequences(const Attn& a, Ctl& ctl)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const uint32_t nan2 = narrow2(nan, nan, T());
    // The good sequence that owns row t, or -1.
    auto owner = [&](int64_t t, Seq* z) {
        int taken, passed;
        const int o = find_seq(a.c.starts, a.c.B, t, lane, &taken, &passed);
        *z = own_seq_of(a.c, o, a.tokens, a.max_chunk);
        return !z->bad && t >= z->start && t - z->start < z->count ? o : -1;
    };
    for (int64_t base = blockIdx.x; base < a.c.B; base += static_cast<int64_t>(gridDim.x) * 32) {
        const int64_t b = base + static_cast<int64_t>(gridDim.x) * lane;
        Seq q{0, 0, 0, 0};
        if (b < a.c.B) q = own_seq_of(a.c, static_cast<int>(b), a.tokens, a.max_chunk);
        if (q.bad && a.status != nullptr && warp == 0) atomicOr(a.status + b, q.bad);
        unsigned m = __ballot_sync(0xFFFFFFFFu, q.bad && q.count > 0);
        while (m != 0) {
            const int i = __ffs(static_cast<int>(m)) - 1;
            m &= m - 1;
            const int64_t t0 = __shfl_sync(0xFFFFFFFFu, q.start, i);
            const int64_t n = __shfl_sync(0xFFFFFFFFu, q.count, i);
            const int64_t words = static_cast<int64_t>(a.Hq) * a.c.D / 2;
            for (int64_t t = t0 + warp; t < t0 + n; t += warps) {
                Seq z;
                if (owner(t, &z) >= 0) continue;
                uint32_t* o = reinterpret_cast<uint32_t*>(a.out) + t * words;
                for (int64_t w = lane; w < words; w += 32) o[w] = nan2;
                if (a.lse != nullptr)
                    for (int w = lane; w < a.Hq; w += 32) a.lse[t * a.Hq + w] = nan;
            }
        }
    }
    bool falls = false;
    for (int64_t b = threadIdx.x; b < a.c.B; b += blockDim.x)
        falls |= a.c.starts[b + 1] < a.c.starts[b];
    if (!__syncthreads_or(falls)) return;
    if (threadIdx.x == 0) ctl.start = Start{0, 0, 0, 0, 0};
    __syncthreads();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp; t < a.tokens;
         t += static_cast<int64_t>(gridDim.x) * warps) {
        Seq z;
        const int b = owner(t, &z);
        if (b < 0) continue;
        const int64_t pos = z.cached + (t - z.start);
        for (int h = 0; h < a.Hq; ++h) {
            float m, l, o[8];
            const bool ok = attend_row<T, E4M3>(a, b, h / a.G, a.q + t * a.q_token + h * a.q_head,
                                                first_key(a, pos), pos + 1, lane, &m, &l, o);
            if (!ok && a.status != nullptr && lane == 0) atomicOr(a.status + b, kBadPage);
            write_row<T>(a, t * a.Hq + h, lane, ok ? m : nan, ok ? l : nan, o);
        }
    }
}

// Output row r of a segment: index of its (token, head) in [tokens, Hq].
__device__ __forceinline__ int64_t out_row(const Attn& a, int q0, int h, int r)
{
    const int t = r / a.G;
    return (static_cast<int64_t>(q0) + t) * a.Hq + h * a.G + (r - t * a.G);
}

// Row r of a segment's item again, key by key, by a warp: to the output or to the
// block's share at `part`.
template <class T, bool E4M3, int DP>
__device__ __noinline__ void again_row(const Tiles& args, const Plan& g, int r, float* part)
{
    const Attn& a = args.a;
    const int lane = threadIdx.x & 31;
    const int64_t origin = static_cast<int64_t>(g.tile0) << kTileShift;
    const int t = (g.row0 + r) / a.G, hq = g.h * a.G + (g.row0 + r - t * a.G);
    const int64_t token = static_cast<int64_t>(g.q0) + t;
    const int64_t lo = origin + max(g.low + t, 0);
    const int64_t hi = min(origin + g.cached + t + 1, origin + (static_cast<int64_t>(g.n) << kTileShift));
    const int64_t orow = token * a.Hq + hq;
    float m, l, o[8];
    attend_row<T, E4M3>(a, g.b, g.h, a.q + token * a.q_token + hq * a.q_head, lo, hi, lane, &m, &l, o);
    if (g.whole) {
        write_row<T>(a, orow, lane, m, l, o);
        return;
    }
    if (lane * 8 < DP) {
        *reinterpret_cast<float4*>(part + lane * 8) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4*>(part + lane * 8 + 4) = make_float4(o[4], o[5], o[6], o[7]);
    }
    if (lane == 0) {
        part[DP] = m;
        part[DP + 1] = l;
    }
}

// Whether row r of a segment sees a position in it whose page is out of range: asked
// only where some page of the segment is.
__device__ __noinline__ bool meets_bad_page(const Attn& a, const Plan& g, int r)
{
    const int64_t origin = static_cast<int64_t>(g.tile0) << kTileShift;
    const int t = (g.row0 + r) / a.G;
    const int64_t hi = origin + min(static_cast<int64_t>(g.cached) + t + 1,
                                    static_cast<int64_t>(g.n) << kTileShift);
    for (int64_t p = origin + max(g.low + t, 0); p < hi;
         p = ((p >> a.c.page_shift) + 1) << a.c.page_shift)
        if (page_of(a.c, g.b, p) < 0) return true;
    return false;
}

// The plan of segment i, or nullptr when there is none or a wait ran out.
template <class Ctl, class Wait>
__device__ __forceinline__ const Plan* plan_at(Ctl& ctl, int i, Wait& wait_all)
{
    if (!wait_all(&ctl.plan_ready[i % kItems], i / kItems)) return nullptr;
    const Plan* p = &ctl.plan[i % kItems];
    return p->n > 0 ? p : nullptr;
}

// Copies of keys (kv = 0) or values (1), by a warp; the keys' warp also plans the
// segments. e4m3: the factors that the codes are multiplied by (FEW: of keys, the
// powers of two themselves; of values, as halves), and with the keys the largest
// exponents of the tile's keys and values (FEW: with the values, of these), plus 256
// where the codes of rows with the factor kUnless have to be looked at. The page of
// tile k + 2 and the exponents of tile k + 1 are on their way while tile k is issued.
template <class T, int DP, bool E4M3, int R, bool SPLIT, bool ALT, int FILL, bool FEW, class Ctl,
          class Wait>
__device__ __forceinline__ void feed(const Tiles& args, Ctl& ctl, const CUtensorMap* map, int kv,
                                     uint32_t stages, uint32_t stage_bytes, uint64_t* fullbar,
                                     uint64_t* emptybar, const Start& start, Wait& wait_all)
{
    const Attn& a = args.a;
    const int lane = threadIdx.x & 31;
    const int P = 1 << a.c.page_shift, box = min(P, kTile);
    const uint32_t box_bytes = E4M3 ? box * a.c.D : box * DP * 2;
    const uint32_t lane_bytes = E4M3 ? lane * 4 * a.c.D : lane * 4 * 128;
    const bool first_of_box = P >= kTile ? lane == 0 : ((lane * 4) & (P - 1)) == 0;
    const uint8_t* exps = kv ? a.c.exps[1] : a.c.exps[0];
    const int64_t exp_step = kv ? a.c.exp_slot_stride[1] : a.c.exp_slot_stride[0];
    const int64_t exp_page = kv ? a.c.exp_page_stride[1] : a.c.exp_page_stride[0];
    Place<FILL> base_at;
    Walk<R> walk(a, start);
    Share sh{};
    int64_t units = start.u0;
    bool ok = true;
    if (kv == 1 && a.gate != nullptr &&
        (a.gate_block < 0 || a.gate_block == static_cast<int>(blockIdx.x))) {
        // Test hook: hold the values until *gate != 0, bounded like every other
        // wait. Nothing sets it in the tests of the timeout path.
        const volatile int32_t* gate = a.gate;
        const long long t0 = clock64();
        while (ok && *gate == 0) {
            __nanosleep(1000);
            ok = clock64() - t0 <= sv::kWaitLimitCycles;
        }
        ok = __all_sync(0xFFFFFFFFu, ok) != 0;
        if (!ok) *reinterpret_cast<volatile int*>(&ctl.stop) = 1;
    }
    for (int item = 0; ok; ++item) {
        const Plan* g;
        if (kv == 0) {
            Segment seg;
            const bool any = walk.next(&seg);
            Plan p{};
            if (any) {
                p = plan_of<SPLIT>(a, seg);
                units += p.n;
                if (p.begins && !p.whole) {
                    // For join_kernel: the item that this block began and did
                    // not finish, and the block that did.
                    const int64_t end = units + (seg.item.hi - seg.t.hi) - 1;  // its last unit
                    int c = blockIdx.x + 1;
                    while (share_begin(start.U, c + 1, gridDim.x) <= end) ++c;
                    sh.leads = 1;
                    sh.b = p.b;
                    sh.h = p.h;
                    sh.row0 = p.row0;
                    sh.rows = p.rows;
                    sh.q0 = p.q0;
                    sh.last = c;
                }
            }
            // (Its place was the plan of kItems segments ago, which the ring
            // of tiles keeps out of everybody's reach.)
            if (lane == 0) {
                ctl.plan[item % kItems] = p;
                sv::mbar_arrive(&ctl.plan_ready[item % kItems]);
            }
            __syncwarp();
            if (!any) break;
            g = &ctl.plan[item % kItems];
        } else if ((g = plan_at(ctl, item, wait_all)) == nullptr) {
            break;
        }
        const int n = g->n, any_lo = g->any_lo, any_hi = g->any_hi, h = g->h;
        const int64_t page_row = g->b * a.c.table_stride +
                                 ((static_cast<int64_t>(g->tile0) << kTileShift) >> a.c.page_shift);
        const int in_page0 =
            static_cast<int>((static_cast<int64_t>(g->tile0) << kTileShift) & (P - 1));
        // The table's entry for this lane's four positions in tile k; INT_MIN
        // if no row sees a position of that page.
        auto entry = [&](int k) {
            const int p = k * kTile + lane * 4 + in_page0;  // from the first tile's page
            const int page0 = (p & ~(P - 1)) - in_page0;
            return k < n && page0 <= any_hi && page0 + P - 1 >= any_lo
                       ? a.c.table[page_row + (p >> a.c.page_shift)]
                       : INT_MIN;
        };
        int v_low = 256, v_high = 0;  // e4m3: the values' exponents so far
        auto good = [&](int32_t page) { return page >= 0 && page < a.c.num_pages; };
        auto slot_of = [&](int k) { return (k * kTile + lane * 4 + in_page0) & (P - 1); };
        struct Exps {
            uint32_t e[4], v[4];  // (v: the values', loaded with the keys)
        };
        const uint8_t* exps_h = exps + (kv ? h * a.c.exp_head_stride[1] : h * a.c.exp_head_stride[0]);
        const uint8_t* v_exps_h = a.c.exps[1] + h * a.c.exp_head_stride[1];
        auto exps_of = [&](int k, int32_t page) {
            Exps x{};
            if (E4M3 && page != INT_MIN) {
                const int64_t pg = good(page) ? page : 0, slot = slot_of(k);
                const uint8_t* e = exps_h + pg * exp_page + slot * exp_step;
#pragma unroll
                for (int i = 0; i < 4; ++i) x.e[i] = e[i * exp_step];
                if (!FEW && kv == 0) {
                    const uint8_t* v = v_exps_h + pg * a.c.exp_page_stride[1] +
                                       slot * a.c.exp_slot_stride[1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.v[i] = v[i * a.c.exp_slot_stride[1]];
                }
            }
            return x;
        };
        int32_t cur = entry(0), next = entry(1);
        Exps xc = exps_of(0, cur);
        Place<FILL> at = base_at;
        if (kv) at.advance(ring_v<ALT>(0, n));
        for (int k = 0; k < n; ++k) {
            const int32_t then = entry(k + 2);
            const Exps xn = exps_of(k + 1, next);
            const bool needed = cur != INT_MIN;
            // A page out of range: page 0 in its place, and NaN for the rows that see
            // a position of it; e4m3: hidden for the others, as what is there would
            // count for the tile's exponents.
            const bool bad = needed && !good(cur);
            if (at.round > 0 && !(ok = wait_all(&emptybar[at.stage], at.round - 1))) break;
            if (bad) {
                cur = 0;
                *reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) = 1;
                if (a.status != nullptr) atomicOr(a.status + g->b, kBadPage);
            }
            if constexpr (E4M3) {
                // Positions that no row sees may hold anything: factor 0, which
                // turns into zeros. So do values that are NaN at positions that
                // not every row sees; these are noted.
                uint32_t top = 0, v_top = 0, f[4], hidden = 0;
                auto note = [&](int p, int times) {
                    const int x = atomicAdd(&ctl.noted[item % kItems], times);
                    if (x < kNoted) ctl.note[item % kItems][x] = p;
                };
                if (bad) {
                    hidden = 15u;
                    xc = Exps{};
                } else if (k < g->inner_lo || k > g->inner_hi) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = k * kTile + lane * 4 + i;
                        const bool outside = p < any_lo || p > any_hi;
                        const bool common = p >= g->all_lo && p <= g->all_hi;
                        if (outside) xc.v[i] = 0;
                        if (outside || (kv == 1 && !common && xc.e[i] == 255u)) {
                            hidden |= 1u << i;
                            if (!outside) note(p, 1);
                            xc.e[i] = 0;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    top = max(top, xc.e[i] == 255u ? 0u : xc.e[i]);
                    if (!FEW && kv == 0) v_top = max(v_top, xc.v[i] == 255u ? 0u : xc.v[i]);
                }
                if (!FEW || kv == 1) top = __reduce_max_sync(0xFFFFFFFFu, top);
                bool apart = false;  // further than float16 holds
                bool looks = false;  // !FEW: some rows' codes have to be looked at
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t e = xc.e[i];
                    f[i] = FEW && kv == 0 ? __float_as_uint(exp_value(e)) : code_factor(e, top);
                    apart |= e > kLeast && e + kSpread < top;
                    if (!FEW && e <= kLeast && (kv == 1 || e + kSpread < top)) {
                        f[i] = both(kUnless);
                        looks = true;
                    }
                }
                if (hidden != 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (hidden >> i & 1u) f[i] = 0;
                }
                if (!FEW) looks = __any_sync(0xFFFFFFFFu, looks) != 0;
                if (FEW && kv == 1 &&
                    min(min(xc.e[0], xc.e[1]), min(xc.e[2], xc.e[3])) <= kLeast) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (xc.e[i] > kLeast || (hidden >> i & 1u)) continue;
                        const uint8_t* codes = a.c.pages[1] + vec_at(a.c, 1, cur, slot_of(k) + i, h);
                        bool any = false;
#pragma unroll 1
                        for (int d = 0; d < a.c.D; d += 16)
                            any |= not_zeros(*reinterpret_cast<const uint4*>(codes + d));
                        if (any) note(0, kNoted + 1);
                    }
                }
                // All rows again (FEW: the keys' codes go into the products as they
                // are, each with a factor of its own; `top` is the lane's).
                if ((apart && (kv == 1 || !FEW)) || (kv == 0 && top > kLarge)) note(0, kNoted + 1);
                if (!FEW && kv == 0) v_top = __reduce_max_sync(0xFFFFFFFFu, v_top);
                if (kv == (FEW ? 1 : 0)) {
                    const int of_values = static_cast<int>(FEW ? top : v_top);
                    if (of_values > static_cast<int>(kLeast)) {
                        v_low = min(v_low, of_values);
                        v_high = max(v_high, of_values);
                        if (lane == 0 && v_high - v_low > kFar) note(0, kNoted + 1);
                    }
                }
                if constexpr (FEW) {
                    if (kv == 0)
                        *reinterpret_cast<uint4*>(&ctl.scale[at.stage][lane * 4]) =
                            make_uint4(f[0], f[1], f[2], f[3]);
                    else
                        *reinterpret_cast<uint2*>(&ctl.scale[at.stage][lane * 2]) = make_uint2(
                            (f[0] & 0xFFFFu) | f[1] << 16, (f[2] & 0xFFFFu) | f[3] << 16);
                } else {
                    *reinterpret_cast<uint4*>(&ctl.factor[at.stage][lane * 4]) =
                        make_uint4(f[0], f[1], f[2], f[3]);
                }
                if constexpr (FEW) {
                    if (kv == 1 && lane == 0) ctl.top[at.stage] = top;
                } else {
                    if (lane == 0) ctl.top[at.stage] = make_uint2(top | (looks ? 256u : 0u), v_top);
                }
                __syncwarp();
            }
            const bool leader = needed && first_of_box;
            const unsigned boxes = __ballot_sync(0xFFFFFFFFu, leader);
            if (lane == 0) {
                ctl.filled[at.stage] = at.round + 1;
                sv::mbar_arrive_expect_tx(&fullbar[at.stage], __popc(boxes) * box_bytes);
            }
            __syncwarp();
            if (leader) {
                const int c1 = slot_of(k);
                const uint32_t to = stages + at.stage * stage_bytes + lane_bytes;
                if (E4M3) {
                    tma_load_4d(to, map, 0, c1, h, cur, &fullbar[at.stage]);
                } else {
#pragma unroll
                    for (int q = 0; q < DP / 64; ++q)
                        tma_load_4d(to + q * kPanel, map, q * 64, c1, h, cur, &fullbar[at.stage]);
                }
            }
            __syncwarp();
            at.advance(kv ? ring_v_step<ALT>(k, n) : ring_k_step<ALT>(k));
            cur = next;
            next = then;
            xc = xn;
        }
        base_at.advance(2 * n);
    }
    if (kv == 0 && lane == 0) {
        sh.units = start.U;
        args.shares[blockIdx.x] = sh;
    }
}

// No copy may be under way when the block ends. Where all waits came to their end
// every tile has been used; where one ran out, whichever it was, the last copies to
// every stage are waited for, whichever warp issued them. All threads come here when
// the roles have met; the block's shared memory stays as long as one of them.
template <int FILL, class Ctl>
__device__ __forceinline__ void land(Ctl& ctl, uint64_t* fullbar)
{
    const int i = threadIdx.x;
    if (ctl.stop != 0 && i < FILL && ctl.filled[i] > 0)
        sv::mbar_wait_bounded(&fullbar[i], (ctl.filled[i] - 1) & 1u, nullptr);
}

// Joins the items that several blocks worked on, in block order: block x takes
// the item that block x of the tile kernel began and did not finish, a warp a
// row. Where a wait ran out in block x, its column fills all outputs with NaN; no
// other column may write then, so each looks at all blocks first (they lie side by
// side: two loads a thread, which the share's covers).
template <class T, int DP>
__global__ void __launch_bounds__(128) join_kernel(const Tiles args, int blocks)
{
    const Attn& a = args.a;
    const int lane = threadIdx.x & 31;
    sv::pdl_wait();
    const Share sh = args.shares[blockIdx.x];
    const bool failed = args.failed[blockIdx.x] != 0;
    bool any_failed = false;
    for (int i = threadIdx.x; i < blocks; i += 128) any_failed |= args.failed[i] != 0;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    if (failed) {
        // A wait ran out: no output of this call can be trusted.
        const int64_t n = static_cast<int64_t>(gridDim.y) * blockDim.x;
        const int64_t i0 = blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x;
        uint32_t* o = reinterpret_cast<uint32_t*>(a.out);
        for (int64_t i = i0; i < a.tokens * a.Hq * a.c.D / 2; i += n) o[i] = narrow2(nan, nan, T());
        if (a.lse != nullptr)
            for (int64_t i = i0; i < a.tokens * a.Hq; i += n) a.lse[i] = nan;
        if (a.status != nullptr)
            for (int64_t i = i0; i < a.c.B; i += n) atomicOr(a.status + i, kTimeout);
        return;
    }
    if (!sh.leads || __syncthreads_or(any_failed)) return;
    const int r = blockIdx.y * (blockDim.x / 32) + (threadIdx.x >> 5);
    if (r >= sh.rows) return;
    constexpr int kPer = DP / 32;
    const float ninf = __uint_as_float(sv::kF32NegInfBits);
    // Shares first .. sh.last, of which some may be empty (fewer units than
    // blocks): 32 at a time, the maxima and sums by a lane each, then the columns.
    float m = ninf, l = 0.f, o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
    const int first = blockIdx.x;
    for (int c0 = first; c0 <= sh.last; c0 += 32) {
        const int c = c0 + lane;
        const int64_t at = ((static_cast<int64_t>(c) * 2 + (c == first ? 1 : 0)) * args.part_rows + r) *
                           (DP + 4);
        const bool has = c <= sh.last &&
                         share_begin(sh.units, c, blocks) < share_begin(sh.units, c + 1, blocks);
        const float pm = has ? args.part[at + DP] : ninf, pl = has ? args.part[at + DP + 1] : 0.f;
        float top = fmaxf(m, pm);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float keep = m == top ? 1.f : sv::ex2(m - top);
        const float w = !has ? 0.f : pm == top ? 1.f : sv::ex2(pm - top);
        l *= keep;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] *= keep;
        unsigned left = __ballot_sync(0xFFFFFFFFu, has);
#pragma unroll 4
        while (left != 0) {
            const int x = __ffs(static_cast<int>(left)) - 1;
            left &= left - 1;
            const float wx = __shfl_sync(0xFFFFFFFFu, w, x);
            const float* from = args.part + __shfl_sync(0xFFFFFFFFu, at, x);
            l = fmaf(__shfl_sync(0xFFFFFFFFu, pl, x), wx, l);
#pragma unroll
            for (int i = 0; i < kPer; ++i) o[i] = fmaf(from[lane + 32 * i], wx, o[i]);
        }
        m = top;
    }
    const int64_t orow = out_row(a, sh.q0, sh.h, sh.row0 + r);
    const float inv = 1.f / l;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int d = lane + 32 * i;
        if (d < a.c.D)
            *reinterpret_cast<uint16_t*>(a.out + (orow * a.c.D + d) * 2) =
                static_cast<uint16_t>(narrow2(o[i] * inv, 0.f, T()));
    }
    if (a.lse != nullptr && lane == 0) a.lse[orow] = fmaf(m, kLn2, logf(l));
}

// Allows `f` its shared memory, once a device.
template <class F>
cudaError_t allow_smem(F* f, size_t smem, std::atomic<uint64_t>* done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit != 0 && (done->load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
    return e;
}

// Launch of join_kernel behind a tile kernel: it may start while that runs and
// waits for it.
template <class T, int DP>
cudaError_t launch_join(const Tiles& t, int blocks, int64_t rows, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks, static_cast<unsigned>((rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, DP>, t, blocks);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled lookup_encode()
{
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        return reinterpret_cast<EncodeTiled>(p);
    return nullptr;
}

// The driver's tensor-map encoder, looked up once.
EncodeTiled encode_fn()
{
    static const EncodeTiled fn = lookup_encode();
    return fn;
}

// Keys (kv = 0) or values (1) as [page][head][slot][element]; a box is the slots
// of one page in one tile, times 64 16-bit elements with the 128-byte swizzle or
// a whole row of codes.
bool make_map(CUtensorMap* map, const Cache& c, int kv, bool f16, bool e4m3, bool swizzled)
{
    const EncodeTiled fn = encode_fn();
    if (fn == nullptr) return false;
    const int P = 1 << c.page_shift;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(P),
                                static_cast<cuuint64_t>(c.Hkv),
                                static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.slot_stride[kv]),
                                   static_cast<cuuint64_t>(c.head_stride[kv]),
                                   static_cast<cuuint64_t>(c.page_stride[kv])};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(e4m3 ? c.D : 64),
                               static_cast<cuuint32_t>(P < kTile ? P : kTile), 1, 1};
    const cuuint32_t unit[4] = {1, 1, 1, 1};
    return fn(map,
              e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                   : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              4, c.pages[kv], dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              !e4m3 ? CU_TENSOR_MAP_SWIZZLE_128B
              : !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE
              : c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Maps, work description and number of blocks of a call. swizzle: e4m3 rows of 128 or
// 64 codes may lie swizzled in shared memory. (The encoder takes every stride that the
// host's checks take, zero among them.)
cudaError_t set_up(const Attn& a, bool f16, bool e4m3, int64_t rows, void* workspace, bool swizzle,
                   CUtensorMap* k, CUtensorMap* v, Tiles* t, int* blocks)
{
    const bool swizzled = swizzle && e4m3 && (a.c.D == 128 || a.c.D == 64);
    if (!make_map(k, a.c, 0, f16, e4m3, swizzled) || !make_map(v, a.c, 1, f16, e4m3, swizzled))
        return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    *blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    *t = Tiles{a,
               reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kShareBytes +
                                        kFailedBytes),
               static_cast<Share*>(workspace),
               reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kShareBytes),
               static_cast<int32_t>(rows),
               swizzled ? 1 : 0};
    return cudaSuccess;
}

}  // namespace
}  // namespace sva
