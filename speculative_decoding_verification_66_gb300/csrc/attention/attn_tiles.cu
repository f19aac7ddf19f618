// attn_tiles.cu -- attention over the paged cache on the 5th-generation tensor
// cores, head sizes up to 128.
//
// For a block of query rows Q and the keys K and values V of a 128-key tile
//   S = Q K^T,  m' = max(m, max S),  P = 2^(c S - m'),
//   l' = l 2^(m - m') + sum P,  O' = O 2^(m - m') + P V,
// with c = scale log2(e): one pass over the cache, the softmax never leaves the
// chip. S, P and O live in tensor memory, a row to a lane: a thread owns a row,
// so the maximum and the sum need no exchange between threads. O is rescaled
// only when the maximum has grown by more than slack() powers of two since the
// last time: the weights stay below 2^slack(), which is what their type holds
// without loss, and hardly any tile after the first needs it.
//
// Two slots, each with its own S, O and softmax warpgroup, take turns on the
// tensor core: while one slot's rows go through the softmax, the other's
// products run.
//   PAIR    an item has up to 256 rows; slot s takes rows 128 s .. and both
//           use every tile of the item.
//   !PAIR   an item has up to 128 rows, both slots hold the same queries and
//           take every second tile; their results are joined at the end.
// PAIR halves the reads of a cache for chunks of more than 128 rows; !PAIR keeps
// the tensor core busy where there are fewer (a draft, a single token).
//
// Warps:
//   0-3, 4-7  softmax of slots 0 and 1 (row = tensor-memory lane = thread), the
//             loads of the queries and the outputs
//   8, 11     issue the products of slots 0 and 1. A warp's later instructions
//             queue behind the products it has issued, so one warp could not
//             look after one slot's barriers while the other's products run.
//   9, 10     load keys and values: page numbers, a bulk tensor copy a page,
//             exponents. Warp 9 also plans the block's segments for all.
//   12-..     helpers (4; e4m3: 8). 16-bit caches: make the values at a tile's hidden
//             positions harmless. e4m3 caches: also expand every tile, exactly,
//             into the stage that the products read.
// The next segment's queries are fetched while the last products of a segment
// run, and its scores begin while the segment's results are written.
//
// Masks. A hidden score is replaced by -inf, whatever it was. A hidden value
// would still be multiplied by a zero weight, and NaN and infinity would come
// through; so in the tiles where some row does not see some position (the ends
// of an item's range), values at positions that not every row sees are
// checked, cleared where they are not finite, and their positions noted; a row
// that does see a noted position is computed again, key by key (attend_row).
// Positions outside the item's range are always cleared: what lies there may
// never have been written.
//
// e4m3. Values are expanded to the query's type, code and exponent, which is
// exact. Keys are expanded to float16 relative to the largest exponent of their
// tile, which multiplies the tile's scores: exact for keys down to 2^-15 of the
// tile's largest, and to 2^-33 of the largest key's magnitude below that, far
// under what float32 keeps of that key's scores. bfloat16 queries become float16
// for this, each row scaled by a power of two that brings its largest element to
// [2^14, 2^15): exact down to 2^-38 of that. float16 takes 25 instructions for 16
// codes, bfloat16 45: the helpers' time is what bounds e4m3 caches.
//
// Work is shared among one block per SM as attn_plan.cuh says; items that
// several blocks share are joined by join_kernel in block order, so results
// depend on the lengths and the number of blocks alone.
#include <climits>
#include <type_traits>

#include "attn_internal.h"
#include "attn_plan.cuh"
#include "tensor_core.cuh"

namespace sva {
namespace {

__device__ __forceinline__ float slack(Bf16) { return 60.f; }
__device__ __forceinline__ float slack(F16) { return 14.f; }  // (below 65504, with 1 to spare)
constexpr int kMaxBlocks = 160;  // shares in the workspace; grids are no larger
constexpr int kNoted = 4;        // noted positions a segment can hold
constexpr int kItems = 16;       // segments whose plans and notes are kept at one time
constexpr size_t kMaxSmem = 232448;

template <int DP, bool E4M3, bool PAIR>
struct Shape {
    static constexpr int kRows = PAIR ? 256 : 128;
    static constexpr int kTileBytes = kTile * DP * 2;  // a K or V tile as the products read it
    static constexpr int kRawBytes = E4M3 ? kTile * DP : 0;
    static constexpr int kQBytes = kRows * DP * 2;
    // Stages in tiles of K or V: what the SM's shared memory holds. (The loads
    // and the notes of hidden values run at most kStages + kRawStages tiles, half
    // as many segments, ahead of the products: well below kItems.)
    static constexpr int kStages = DP == 128 ? (E4M3 ? 3 : (PAIR ? 5 : 6)) : (E4M3 ? 4 : 8);
    static constexpr int kRawStages = E4M3 ? (DP == 128 ? (PAIR ? 3 : 5) : 8) : 0;
    static_assert((kStages + kRawStages) / 2 + 1 < kItems - 2, "notes");
    static constexpr int kHelpers = E4M3 ? 8 : 4;
    static constexpr int kThreads = (12 + kHelpers) * 32;
    // e4m3: registers a thread of the softmax warps and of the others; together
    // no more than the 640 threads are launched with, 96 each.
    static constexpr int kRegsRow = 128, kRegsOther = 72, kRegsLaunch = 96;
    static_assert(8 * kRegsRow + 12 * kRegsOther <= 20 * kRegsLaunch, "registers");
    static constexpr int kPanel = kTile * 128;  // bytes of 64 elements of every row
    static constexpr int kTiles = kQBytes + kStages * kTileBytes + kRawStages * kRawBytes;
};

// A segment as the warps need it. Positions count from the segment's first
// tile; tiles are numbered from it.
struct Plan {
    int32_t n;                         // tiles; 0: no more segments
    int32_t b, h, q0, row0, rows;
    int32_t tile0;                     // the first tile's number in the sequence
    int32_t cached;                    // row r stands at position cached + r / G
    int32_t lo0, hi0, lo1, hi1;        // PAIR: tiles of either slot
    int32_t any_lo, any_hi;            // positions that some row sees
    int32_t all_lo, all_hi;            // positions that every row sees
    int32_t inner_lo, inner_hi;        // tiles wholly in `all`; the others have hidden values
    int32_t begins, whole;             // the item begins here; is all here
};

// Shared memory besides the tiles.
template <int STAGES, int RAW, bool PAIR>
struct Control {
    uint64_t full[STAGES], empty[STAGES], fixed[STAGES];
    uint64_t raw_full[RAW > 0 ? RAW : 1], raw_empty[RAW > 0 ? RAW : 1];
    uint64_t s_full[2], p_ready[2], q_ready, q_free, o_full, o_free, s_free, ml_ready, done;
    uint64_t plan_ready[kItems];
    uint32_t tmem;
    int stop;
    int burst;  // PAIR: a slot's products are under way
    Start start;
    int64_t sums[20];
    Plan plan[kItems];
    int noted[kItems];             // how many positions are noted
    int note[kItems][kNoted];      // which, counted as in the plan
    int bad_page[kItems];
    // e4m3: powers of two that the rows of this segment and the next are divided by
    float q_scale[2][RAW > 0 ? (PAIR ? 256 : 128) : 1];
    float k_scale[4];  // .. and of the keys of the last four tiles
    // e4m3, for every raw stage: a row's factor (two 16-bit halves), the largest
    // exponent (keys), whether some row needs two factors (values), exponents.
    alignas(16) uint32_t factor[RAW > 0 ? RAW : 1][RAW > 0 ? kTile : 4];
    uint32_t top[RAW > 0 ? RAW : 1], two[RAW > 0 ? RAW : 1];
    uint8_t exps[RAW > 0 ? RAW : 1][RAW > 0 ? kTile : 4];
};

struct Tiles {
    Attn a;
    float* part;   // [blocks][2][rows][part_cols]: unnormalised O, then m and l
    Share* shares; // [blocks]
    int32_t part_rows;
    // A tile in shared memory: rows of 128 bytes (64 elements), eight to a
    // group; bytes from a group to the next, and to the next 64 elements.
    int32_t group, panel;
    // Copies of whole 128-element rows: pages and heads are one axis, a page
    // page_heads steps, a head head_step. 0: a copy for each 64 elements.
    int32_t page_heads, head_step;
};

// Where the tiles of a segment lie in the ring: the order in which the products
// use them. PAIR: K0 V0 K1 V1 ..; otherwise K0 K1 V0 K2 V1 .., since the second
// slot's scores come before the first slot's values.
template <bool PAIR>
__device__ __forceinline__ int ring_v(int k, int n)
{
    return PAIR ? 2 * k + 1 : (k == n - 1 ? 2 * k + 1 : 2 * k + 2);
}
// From a tile's keys, and its values, to the next tile's.
template <bool PAIR>
__device__ __forceinline__ int ring_k_step(int k)
{
    return !PAIR && k == 0 ? 1 : 2;
}
template <bool PAIR>
__device__ __forceinline__ int ring_v_step(int k, int n)
{
    return !PAIR && k == n - 2 ? 1 : 2;
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

__device__ __forceinline__ int clamp32(int64_t v)
{
    return static_cast<int>(max(min(v, int64_t(INT_MAX / 2)), int64_t(INT_MIN / 2)));
}

template <bool PAIR>
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
    if (PAIR) {
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
// Expanding e4m3. A value is code 2^(e - 127). bfloat16: the code's exponent
// and mantissa bits, moved under bfloat16's wider exponent, read as the value
// times 2^-120 (the biases differ by 127 - 7; subnormal codes land on subnormal
// bfloat16s), so one multiplication by 2^(e - 7) gives the value exactly; it
// takes two where that exceeds bfloat16. float16: the conversion instruction,
// then one multiplication by 2^(e - 127), two where that is not a normal
// float16. Either way two values an instruction.
// ---------------------------------------------------------------------------
struct Factor {
    uint32_t f1, f2;  // both halves alike
    bool two;
};
__device__ __forceinline__ uint32_t both(uint32_t h) { return h | (h << 16); }
__device__ __forceinline__ Factor factor_of(uint32_t e, Bf16)
{
    const uint32_t x = min(e, 134u), y = e == 255u ? 0u : e - x;
    return Factor{e == 255u ? both(0x7FFFu) : (x + 120u) * 0x00800080u, (y + 127u) * 0x00800080u,
                  y != 0};
}
__device__ __forceinline__ Factor factor_of(uint32_t e, F16)
{
    if (e == 255u) return Factor{both(0x7FFFu), both(0x3C00u), false};
    const int x = static_cast<int>(e) - 127;
    const int g = min(max(x, -14), 15), h = x - g;
    const uint32_t second = h < -24 ? 0u : h < -14 ? 1u << (h + 24) : (h > 15 ? 30u : h + 15u) << 10;
    return Factor{both(static_cast<uint32_t>(g + 15) << 10), both(second), h != 0};
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b, Bf16)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b, F16)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Four codes to two words of 16-bit values, before the factor.
__device__ __forceinline__ uint2 spread(uint32_t w, Bf16)
{
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    return make_uint2((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u),
                      (b & 0x80008000u) | ((b >> 4) & 0x07F007F0u));
}
__device__ __forceinline__ uint2 spread(uint32_t w, F16)
{
    return make_uint2(e4m3_to_f16x2(w & 0xFFFFu), e4m3_to_f16x2(w >> 16));
}
// Factor of a key's codes relative to the tile's largest exponent.
__device__ __forceinline__ uint32_t key_factor(uint32_t e, uint32_t top)
{
    if (e == 255u) return both(0x7FFFu);
    const int d = static_cast<int>(top) - static_cast<int>(e);
    return both(d <= 14 ? static_cast<uint32_t>(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u);
}
// 16 codes times a factor, as sixteen 16-bit values.
template <class T>
__device__ __forceinline__ void expand(uint4 codes, uint32_t f, uint32_t (&o)[8])
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint2 s = spread(w[i], T());
        o[2 * i] = mul2(s.x, f, T());
        o[2 * i + 1] = mul2(s.y, f, T());
    }
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
// Byte offset of 16-byte chunk `chunk` of a row in a tile with the 128-byte
// swizzle (group and panel: see Tiles).
__device__ __forceinline__ uint32_t tile_chunk(int row, int chunk, int group, int panel)
{
    return (row >> 3) * group + (chunk >> 3) * panel + (row & 7) * 128 +
           (((chunk & 7) ^ (row & 7)) << 4);
}

// Sum of int64 over the block; every thread gets it.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* sums, int warps)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t t = 0;
    for (int w = 0; w < warps; ++w) t += sums[w];
    return t;
}

// Rows of sequences whose lengths are bad become NaN; block c of n takes
// sequences c, c + n, ..
template <class T>
__device__ void refuse_sequences(const Attn& a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint32_t nan2 = narrow2(__uint_as_float(0x7FFFFFFFu), __uint_as_float(0x7FFFFFFFu), T());
    for (int64_t base = blockIdx.x; base < a.c.B; base += static_cast<int64_t>(gridDim.x) * 32) {
        const int64_t b = base + static_cast<int64_t>(gridDim.x) * lane;
        Seq q{0, 0, 0, 0};
        if (b < a.c.B) q = seq_of(a.c, static_cast<int>(b), a.tokens, a.max_chunk);
        if (q.bad && a.status != nullptr && warp == 0) atomicOr(a.status + b, q.bad);
        unsigned m = __ballot_sync(0xFFFFFFFFu, q.bad && q.count > 0);
        while (m != 0) {
            const int i = __ffs(static_cast<int>(m)) - 1;
            m &= m - 1;
            const int64_t t0 = __shfl_sync(0xFFFFFFFFu, q.start, i);
            const int64_t n = __shfl_sync(0xFFFFFFFFu, q.count, i);
            const int64_t words = n * a.Hq * a.c.D / 2, w0 = t0 * a.Hq * a.c.D / 2;
            uint32_t* o = reinterpret_cast<uint32_t*>(a.out);
            for (int64_t w = warp * 32 + lane; w < words; w += warps * 32) o[w0 + w] = nan2;
            if (a.lse != nullptr)
                for (int64_t w = warp * 32 + lane; w < n * a.Hq; w += warps * 32)
                    a.lse[t0 * a.Hq + w] = __uint_as_float(0x7FFFFFFFu);
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
    const int64_t pos = origin + g.cached + t, token = static_cast<int64_t>(g.q0) + t;
    const int64_t lo = max(first_key(a, pos), origin);
    const int64_t hi = min(pos + 1, origin + (static_cast<int64_t>(g.n) << kTileShift));
    const int64_t orow = token * a.Hq + hq;
    float m, l, o[8];
    attend_row<T, E4M3>(a, g.b, g.h, a.q + token * a.q_token + hq * a.q_head, lo, hi, lane, &m, &l, o);
    if (g.whole) {
        const float x = 1.f / l;
        if (lane * 8 < a.c.D)
            *reinterpret_cast<uint4*>(a.out + (orow * a.c.D + lane * 8) * 2) =
                make_uint4(narrow2(o[0] * x, o[1] * x, T()), narrow2(o[2] * x, o[3] * x, T()),
                           narrow2(o[4] * x, o[5] * x, T()), narrow2(o[6] * x, o[7] * x, T()));
        if (a.lse != nullptr && lane == 0) a.lse[orow] = fmaf(m, kLn2, logf(l));
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

template <class T, int DP, bool E4M3, bool PAIR>
__global__ void __launch_bounds__(Shape<DP, E4M3, PAIR>::kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ Tiles args)
{
    using X = Shape<DP, E4M3, PAIR>;
    constexpr int S = X::kStages, RS = X::kRawStages, R = X::kRows;
    constexpr int kFill = E4M3 ? RS : S;  // stages that the copies fill
    const Attn& a = args.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    Control<S, RS, PAIR>& ctl = *reinterpret_cast<Control<S, RS, PAIR>*>(smem + X::kTiles);
    const uint32_t base = sv::smem_addr(smem);
    const uint32_t sq = base, st = base + X::kQBytes, sr = st + S * X::kTileBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kWarps = X::kThreads / 32;

    sv::pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            sv::mbar_init(&ctl.full[i], E4M3 ? X::kHelpers : 1);
            // Both slots' products and, for 16 bits, the helpers pass every tile
            // in order, used or not: else a parity could stand for another round
            // of the stage than they mean.
            sv::mbar_init(&ctl.empty[i], E4M3 ? 2 : 2 + X::kHelpers);
            sv::mbar_init(&ctl.fixed[i], X::kHelpers);
        }
        for (int i = 0; i < RS; ++i) {
            sv::mbar_init(&ctl.raw_full[i], 1);
            sv::mbar_init(&ctl.raw_empty[i], X::kHelpers);
        }
        for (int i = 0; i < 2; ++i) {
            sv::mbar_init(&ctl.s_full[i], 1);
            sv::mbar_init(&ctl.p_ready[i], 4);
        }
        sv::mbar_init(&ctl.q_ready, 8);
        sv::mbar_init(&ctl.o_full, 2);
        sv::mbar_init(&ctl.ml_ready, 8);
        sv::mbar_init(&ctl.q_free, 2);
        sv::mbar_init(&ctl.o_free, 8);
        sv::mbar_init(&ctl.s_free, 8);
        sv::mbar_init(&ctl.done, 2);
        for (int i = 0; i < kItems; ++i) sv::mbar_init(&ctl.plan_ready[i], 1);
        // (The swizzle needs tiles on 1024-byte boundaries. There is no static
        // shared memory before them, so they are; if not, the call fails.)
        ctl.burst = 0;
        ctl.stop = (base & 1023u) != 0;
        for (int i = 0; i < kItems; ++i) ctl.noted[i] = ctl.bad_page[i] = 0;
        sv::fence_barrier_init();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         sv::smem_addr(&ctl.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }

    // Where this block starts.
    {
        const int tid = threadIdx.x;
        int64_t mine = 0, first = 0;
        for (int64_t b = tid; b < a.c.B; b += X::kThreads) {
            const Seq q = seq_of(a.c, static_cast<int>(b), a.tokens, a.max_chunk);
            const int64_t u = head_units<R>(a, q) * a.c.Hkv;
            if (b == tid) first = u;
            mine += u;
        }
        const int64_t U = block_sum(mine, ctl.sums, kWarps);
        const int64_t u0 = share_begin(U, blockIdx.x, gridDim.x);
        const int64_t u1 = share_begin(U, blockIdx.x + 1, gridDim.x);
        if (tid == 0) ctl.start = Start{u0, u1, U, 0, 0};
        __syncthreads();
        if (u0 < u1) {
            int64_t before = 0;
            for (int64_t base_b = 0; base_b < a.c.B && before <= u0; base_b += X::kThreads) {
                const int64_t b = base_b + tid;
                int64_t u = first;
                if (base_b > 0)
                    u = b < a.c.B ? head_units<R>(a, seq_of(a.c, static_cast<int>(b), a.tokens,
                                                            a.max_chunk)) * a.c.Hkv
                                  : 0;
                int64_t scan = u;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, scan, d);
                    if (lane >= d) scan += o;
                }
                __syncthreads();
                if (lane == 31) ctl.sums[warp] = scan;
                __syncthreads();
                int64_t chunk = 0;
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) scan += ctl.sums[w];
                    chunk += ctl.sums[w];
                }
                const int64_t begin = before + scan - u;
                if (u0 >= begin && u0 < begin + u) {
                    ctl.start.off = u0 - begin;
                    ctl.start.b = static_cast<int32_t>(b);
                }
                before += chunk;
            }
        }
        refuse_sequences<T>(a);
    }
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl.tmem;
    const Start start = ctl.start;
    volatile int* stop = &ctl.stop;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (sv::mbar_wait_bounded(bar, parity & 1u, stop)) return true;
        *stop = 1;
        return false;
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0;
    };
    int item = 0;  // segments taken so far
    // The next segment's plan, or nullptr when there is none or a wait ran out.
    auto plan_at = [&](int i) -> const Plan* {
        if (!wait_all(&ctl.plan_ready[i % kItems], i / kItems)) return nullptr;
        const Plan* p = &ctl.plan[i % kItems];
        return p->n > 0 ? p : nullptr;
    };

    if (warp < 8) {
        // ------------------------------------------------------------------
        // Softmax of slot s; thread = row.
        // ------------------------------------------------------------------
        if (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(X::kRegsRow));
        const int s = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t s_addr = lane_base + s * 128, o_addr = lane_base + 256 + s * DP;
        const float ninf = __uint_as_float(sv::kF32NegInfBits);
        const int slot_row = PAIR ? 128 * s + row : row;  // row of the item
        const int warp_row = slot_row - lane;
        uint32_t tiles_done = 0;
        int tiles_before = 0;  // of the segments before, for the keys' exponents

        // Queries of a segment: PAIR: the slot's 128 rows; otherwise half of the
        // item's rows each slot. Fetched into registers first, stored when the
        // products of the segment before have read theirs: panels of 64
        // elements, swizzled, zeros past D.
        constexpr int kChunks = DP / 8, kCount = PAIR ? 128 : 64;
        constexpr int kFetch = kCount * kChunks / 128;
        uint4 qv[kFetch];
        const int first = (threadIdx.x & 127) / kChunks + (PAIR ? 128 * s : 64 * s);
        const int ch = threadIdx.x % kChunks;
        auto fetch = [&](const Plan& x) {
#pragma unroll
            for (int i = 0; i < kFetch; ++i) {
                const int r = first + i * (128 / kChunks);
                qv[i] = make_uint4(0, 0, 0, 0);
                if (r < x.rows && ch * 8 < a.c.D) {
                    const int rr = x.row0 + r, t = rr / a.G;
                    qv[i] = *reinterpret_cast<const uint4*>(
                        a.q + (static_cast<int64_t>(x.q0) + t) * a.q_token +
                        static_cast<int64_t>(x.h * a.G + (rr - t * a.G)) * a.q_head + ch * 16);
                }
            }
        };
        auto store = [&](const Plan& x, int at) {
#pragma unroll
            for (int i = 0; i < kFetch; ++i) {
                const int r = first + i * (128 / kChunks);
                const bool has = r < x.rows;
                if constexpr (E4M3 && std::is_same<T, Bf16>::value) {
                    // To float16, scaled. The kChunks lanes of a row are neighbours.
                    const uint32_t u[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                    uint32_t top = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top = max(top, max(u[k] << 16 & 0x7FFF0000u, u[k] & 0x7FFF0000u));
#pragma unroll
                    for (int d = kChunks / 2; d > 0; d >>= 1)
                        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    // 2^(14 - exponent), at most 2^126
                    const int e = max(static_cast<int>(top >> 23), 15);
                    const float up = __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = narrow2(sv::bf16_lo(u[k]) * up, sv::bf16_hi(u[k]) * up, F16());
                    qv[i] = make_uint4(h[0], h[1], h[2], h[3]);
                    if (has && ch == 0)
                        ctl.q_scale[at & 1][r] =
                            __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
                }
                if (has)
                    st_shared_v4(sq + (r >> 7) * (128 * DP * 2) +
                                     tile_chunk(r & 127, ch, 1024, X::kPanel),
                                 qv[i]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) sv::mbar_arrive(&ctl.q_ready);
        };

        const Plan* ahead = plan_at(0);
        if (ahead != nullptr) {
            fetch(*ahead);
            store(*ahead, 0);
        }
        bool ok = true;
        for (; ahead != nullptr; ++item) {
            const Plan& g = *ahead;
            const int rows = g.rows;
            const bool live = warp_row < rows;  // some row of this warp exists
            float m = ninf, l = 0.f;
            bool begun = false;
            {
                // The last position that the row sees, and the first.
                const int pos = g.cached + (g.row0 + min(slot_row, rows - 1)) / a.G;
                const int low = a.window > 0 ? pos - static_cast<int>(a.window) + 1 : INT_MIN / 2;
                const int k0 = PAIR ? (s ? g.lo1 : g.lo0) : s;
                const int k1 = PAIR ? (s ? g.hi1 : g.hi0) : g.n;
                float row_c = a.scale_log2, c = row_c;
                for (int k = k0; k < k1; k += PAIR ? 1 : 2) {
                    if (!(ok = wait_all(&ctl.s_full[s], tiles_done))) break;
                    ++tiles_done;
                    if (live) {
                        fence_after();
                        if (E4M3 && std::is_same<T, Bf16>::value && !begun)
                            row_c = a.scale_log2 * ctl.q_scale[item & 1][min(slot_row, rows - 1)];
                        const int clo = low - k * kTile, chi = pos - k * kTile;
                        const bool masked =
                            __any_sync(0xFFFFFFFFu, clo > 0 || chi < kTile - 1) != 0;
                        // The loops below are kept rolled: all roles' code has to
                        // stay in the instruction caches.
                        if (E4M3) c = row_c * ctl.k_scale[(tiles_before + k) & 3];
                        if (masked) {
#pragma unroll 1
                            for (int x = 0; x < kTile; x += 16) {
                                float v[16];
                                tmem_ld(s_addr + x, v);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    v[i] = x + i >= clo && x + i <= chi ? v[i] : ninf;
                                tmem_st(s_addr + x, v);
                            }
                            tmem_wait_st();
                        }
                        float v[32], mt = ninf;
#pragma unroll 1
                        for (int x = 0; x < kTile; x += 32) mt = fmaxf(mt, tmem_ld_max(s_addr + x, v));
                        // (scale > 0; a NaN score is left out here and comes through below)
                        mt *= c;
                        const bool grow = mt > m + slack(T()) || (!begun && mt > m);
                        if (begun && __any_sync(0xFFFFFFFFu, grow)) {
                            // The slot's products so far are complete: s_full's
                            // commit came after them.
                            const float keep = grow ? sv::ex2(m - mt) : 1.f;
#pragma unroll 1
                            for (int x = 0; x < DP / 16; ++x) {
                                float o[16];
                                tmem_ld(o_addr + 16 * x, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= keep;
                                tmem_st(o_addr + 16 * x, o);
                            }
                            l *= keep;
                        }
                        if (grow) m = mt;
                        begun = true;
                        const float shift = m == ninf ? 0.f : -m;
                        float2 l0 = make_float2(0.f, 0.f), l1 = l0;
                        // The weights, the last 32 columns first: they take the
                        // columns of the upper half from the top.
#pragma unroll 1
                        for (int x = kTile - 32;;) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float2 p = fma2(make_float2(v[2 * i], v[2 * i + 1]), c, shift);
                                float2 q = fma2(make_float2(v[2 * i + 2], v[2 * i + 3]), c, shift);
                                p = make_float2(sv::ex2(p.x), sv::ex2(p.y));
                                q = make_float2(sv::ex2(q.x), sv::ex2(q.y));
                                l0 = add2(l0, p);
                                l1 = add2(l1, q);
                                w[i] = narrow2(p.x, p.y, T());
                                w[i + 1] = narrow2(q.x, q.y, T());
                            }
                            tmem_st(s_addr + 64 + x / 2, w);
                            if (x == 0) break;
                            x -= 32;
                            tmem_ld(s_addr + x, v);
                        }
                        l += (l0.x + l0.y) + (l1.x + l1.y);
                        tmem_wait_st();
                        fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) sv::mbar_arrive(&ctl.p_ready[s]);
                }
            }
            if (!ok) break;

            // --------------------------------------------------------------
            // The rows' results.
            // --------------------------------------------------------------
            const int n = g.n;
            tiles_before += n;
            ahead = plan_at(item + 1);
            if (ahead != nullptr) {
                fetch(*ahead);
                if (!(ok = wait_all(&ctl.q_free, item))) break;
                store(*ahead, item + 1);
            }
            if (!(ok = wait_all(&ctl.o_full, item))) break;
            fence_after();
            float w0 = 1.f, w1 = 0.f;
            if (!PAIR) {
                // The slots exchange their rows' maxima and sums through the
                // scores' columns, which the products have done with.
                if (live) {
                    tmem_st2(s_addr, m, l);
                    tmem_wait_st();
                    fence_before();
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.ml_ready);
                if (!(ok = wait_all(&ctl.ml_ready, item))) break;
                if (live) {
                    fence_after();
                    float om, ol;
                    tmem_ld2(lane_base + (1 - s) * 128, om, ol);
                    fence_before();
                    const float top = fmaxf(m, om);
                    const float wm = m == top ? 1.f : sv::ex2(m - top);
                    const float wo = om == top ? 1.f : sv::ex2(om - top);
                    w0 = s ? wo : wm;
                    w1 = s ? wm : wo;
                    // (the same order in both slots)
                    l = (s ? ol : l) * w0 + (s ? l : ol) * w1;
                    m = top;
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.s_free);
            }
            const bool whole = g.whole != 0, valid = slot_row < rows;
            // A row that sees a noted position is computed again below.
            const int noted = *reinterpret_cast<volatile int*>(&ctl.noted[item % kItems]);
            const bool bad = *reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) != 0;
            const int r = g.row0 + min(slot_row, rows - 1), token = r / a.G;
            bool again = noted > kNoted;
            if (noted > 0) {
                const int pos = g.cached + token;
                const int low = a.window > 0 ? pos - static_cast<int>(a.window) + 1 : INT_MIN / 2;
                for (int i = 0; i < min(noted, kNoted); ++i) {
                    const int p = *reinterpret_cast<volatile int*>(&ctl.note[item % kItems][i]);
                    again |= p >= low && p <= pos;
                }
            }
            again = again && valid && !bad;
            const float nan = __uint_as_float(0x7FFFFFFFu);
            float* share = args.part + (static_cast<int64_t>(blockIdx.x) * 2 + (g.begins ? 1 : 0)) *
                                           args.part_rows * (DP + 4);
            if (live) {
                // Columns of the row, kCols at a time: all, or the slot's half
                // where both slots hold the row.
                constexpr int kCols = PAIR ? 64 : DP / 2;
                const int64_t orow = (static_cast<int64_t>(g.q0) + token) * a.Hq + g.h * a.G +
                                     (r - token * a.G);
                const float inv = bad ? nan : (whole ? 1.f / l : 1.f);
                float* part = share + static_cast<int64_t>(slot_row) * (DP + 4);
#pragma unroll 1
                for (int x = 0; x < (PAIR ? DP / 64 : 1); ++x) {
                    const int k0 = PAIR ? 64 * x : s * kCols;
                    float o[kCols];
                    __syncwarp();
                    if constexpr (PAIR) {
                        tmem_ld(o_addr + k0, o);
                        if (!begun) {
#pragma unroll
                            for (int i = 0; i < kCols; ++i) o[i] = 0.f;
                        }
                    } else {
                        float p[kCols];
                        // (slot 1 without a tile: its columns are read and not used)
                        tmem_ld(lane_base + 256 + k0, o, lane_base + 256 + DP + k0, p);
#pragma unroll
                        for (int i = 0; i < kCols; ++i) o[i] = n > 1 ? o[i] * w0 + p[i] * w1 : o[i];
                    }
                    if (!valid || again) continue;
#pragma unroll
                    for (int i = 0; i < kCols; ++i) o[i] *= inv;
                    if (whole) {
                        uint8_t* to = a.out + (orow * a.c.D + k0) * 2;
#pragma unroll
                        for (int i = 0; i < kCols; i += 8)
                            if (k0 + i < a.c.D)
                                *reinterpret_cast<uint4*>(to + i * 2) =
                                    make_uint4(narrow2(o[i], o[i + 1], T()),
                                               narrow2(o[i + 2], o[i + 3], T()),
                                               narrow2(o[i + 4], o[i + 5], T()),
                                               narrow2(o[i + 6], o[i + 7], T()));
                    } else {
#pragma unroll
                        for (int i = 0; i < kCols; i += 4)
                            *reinterpret_cast<float4*>(part + k0 + i) =
                                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                if (valid && !again && (PAIR || s == 0)) {
                    if (!whole) {
                        part[DP] = m;
                        part[DP + 1] = bad ? nan : l;
                    } else if (a.lse != nullptr) {
                        a.lse[orow] = bad ? nan : fmaf(m, kLn2, logf(l));
                    }
                }
                __syncwarp();
                unsigned todo = PAIR || s == 0 ? __ballot_sync(0xFFFFFFFFu, again) : 0u;
                while (todo != 0) {
                    const int i = __ffs(static_cast<int>(todo)) - 1;
                    todo &= todo - 1;
                    again_row<T, E4M3, DP>(args, g, warp_row + i,
                                           share + static_cast<int64_t>(warp_row + i) * (DP + 4));
                }
                fence_before();
            }
            // The notes of two segments before: their readers have all come to
            // this one since, and the segment that gets their place is still out
            // of the loads' reach.
            __syncwarp();
            if (threadIdx.x == 0) {
                ctl.noted[(item + kItems - 2) % kItems] = 0;
                ctl.bad_page[(item + kItems - 2) % kItems] = 0;
            }
            if (lane == 0) sv::mbar_arrive(&ctl.o_free);
        }
    } else {
    if (E4M3) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kRegsOther));
    if (warp == 8 || warp == 11) {
        // ------------------------------------------------------------------
        // Products of slot s: the warp stays together, one lane issues. It
        // passes every tile in ring order, its own and the other slot's.
        // ------------------------------------------------------------------
        using TS = typename std::conditional<E4M3, F16, T>::type;
        constexpr uint32_t id_s = idesc<TS, kTile, false>(), id_o = idesc<T, DP, true>();
        const int s = warp == 8 ? 0 : 1;
        const uint64_t dq = smem_desc(sq + (PAIR ? s * (128 * DP * 2) : 0), 16, 1024);
        const uint64_t dk = smem_desc(st, 16, args.group), dv = smem_desc(st, args.panel, args.group);
        const uint32_t panel = args.panel >> 4, v_step = args.group >> 3;  // 16 keys: two groups
        const uint32_t s_addr = tmem + s * 128, o_addr = tmem + 256 + s * DP;
        Place<S> at;
        uint32_t fixes = 0, tiles = 0;
        bool ok = true;
        for (; ok; ++item) {
            const Plan* g = plan_at(item);
            if (g == nullptr || !(ok = wait_all(&ctl.q_ready, item))) break;
            const int n = g->n, inner_lo = g->inner_lo, inner_hi = g->inner_hi;
            const int k0 = PAIR ? (s ? g->lo1 : g->lo0) : s, k1 = PAIR ? (s ? g->hi1 : g->hi0) : n;
            // !PAIR: the slots have exchanged their rows' sums of the segment
            // before, through the scores' columns.
            if (!PAIR && item > 0 && !(ok = wait_all(&ctl.s_free, item - 1))) break;
            bool begun = false;
            int kk = 0, vv = 0, left = k1 <= k0 ? 0 : PAIR ? k1 - k0 : (k1 - k0 + 1) / 2;
            if (left == 0 && lane == 0) sv::mbar_arrive(&ctl.q_free);
            for (int i = 0; i < 2 * n; ++i) {
                const bool is_v = vv < n && ring_v<PAIR>(vv, n) == i;
                const int k = is_v ? vv++ : kk++;
                const bool mine = k >= k0 && k < k1 && (PAIR || ((k - k0) & 1) == 0);
                const bool edge = !E4M3 && is_v && (k < inner_lo || k > inner_hi);
                if (!(ok = wait_all(&ctl.full[at.stage], at.round))) break;
                Place<S> keys = at;
                bool scores = mine && !is_v;
                if (mine && is_v) {
                    if (edge && !(ok = wait_all(&ctl.fixed[at.stage], fixes >> at.stage))) break;
                    // (the results before have been read)
                    if (!begun && item > 0 && !(ok = wait_all(&ctl.o_free, item - 1))) break;
                    // The slot's next keys are next in the ring. Where they are there
                    // already their scores follow at once: looking at a barrier
                    // between the two would let the tensor core run dry.
                    keys.advance(1);
                    for (int x = 0; x < 2; ++x) {
                        if (left > 0 && !scores)
                            scores = __all_sync(0xFFFFFFFFu, mbar_test(&ctl.full[keys.stage],
                                                                       keys.round & 1u));
                        if (x == 0 && !(ok = wait_all(&ctl.p_ready[s], tiles))) break;
                    }
                    if (!ok) break;
                    ++tiles;
                    if (PAIR) {
                        // One slot's products after the other's: side by side both
                        // would end late, and both softmaxes would then run while
                        // the tensor core idles.
                        const long long t0 = clock64();
                        bool got;
                        do {
                            got = __any_sync(0xFFFFFFFFu,
                                             lane == 0 && atomicCAS(&ctl.burst, 0, 1) == 0) != 0;
                        } while (!got && __all_sync(0xFFFFFFFFu, *stop == 0 && clock64() - t0 <
                                                                                  sv::kWaitLimitCycles));
                        if (!(ok = got)) {
                            *stop = 1;
                            break;
                        }
                    }
                }
                fence_after();
                if (mine) {
                    if (elect_one()) {
                        if (is_v) {
                            const uint64_t b = dv + at.stage * (X::kTileBytes >> 4);
#pragma unroll
                            for (int x = 0; x < kTile / 16; ++x)
                                mma_ts(o_addr, s_addr + 64 + x * 8, b + x * v_step, id_o,
                                       begun || x > 0);
                            mma_commit(&ctl.empty[at.stage]);
                        }
                        if (scores) {
                            const uint64_t b = dk + keys.stage * (X::kTileBytes >> 4);
#pragma unroll
                            for (int x = 0; x < DP / 16; ++x) {
                                const uint32_t o = (x & 3) * 2;
                                mma_ss(s_addr, dq + o + (x >> 2) * (X::kPanel >> 4),
                                       b + o + (x >> 2) * panel, id_s, x > 0);
                            }
                            mma_commit(&ctl.s_full[s]);
                            mma_commit(&ctl.empty[keys.stage]);
                            if (left == 1) mma_commit(&ctl.q_free);
                        }
                        if (PAIR && is_v) atomicExch(&ctl.burst, 0);
                    }
                    __syncwarp();
                    begun |= is_v;
                    left -= scores;
                } else if (lane == 0) {
                    sv::mbar_arrive(&ctl.empty[at.stage]);
                }
                if (edge) fixes ^= 1u << at.stage;
                if (is_v && scores) {
                    ++kk;
                    ++i;
                    at.advance(1);
                }
                at.advance(1);
            }
            if (!ok) break;
            if (elect_one()) mma_commit(&ctl.o_full);
            __syncwarp();
        }
        // Everything issued has completed once both have arrived.
        if (elect_one()) mma_commit(&ctl.done);
        __syncwarp();
        sv::mbar_wait_bounded(&ctl.done, 0, nullptr);
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------------
        // Copies of keys (warp 9, which also plans the segments) and values
        // (warp 10). The page of tile k + 2 and the exponents of tile k + 1 are
        // on their way while tile k is issued.
        // ------------------------------------------------------------------
        const int kv = warp - 9;
        const CUtensorMap* map = kv ? &vmap : &kmap;
        uint64_t* fullbar = E4M3 ? ctl.raw_full : ctl.full;
        uint64_t* emptybar = E4M3 ? ctl.raw_empty : ctl.empty;
        const int P = 1 << a.c.page_shift, box = min(P, kTile);
        const uint32_t box_bytes = E4M3 ? box * a.c.D : box * DP * 2;
        const uint32_t lane_bytes = E4M3 ? lane * 4 * a.c.D : lane * 4 / 8 * args.group;
        const bool first_of_box = P >= kTile ? lane == 0 : ((lane * 4) & (P - 1)) == 0;
        const uint8_t* exps = kv ? a.c.exps[1] : a.c.exps[0];
        const int64_t exp_step = kv ? a.c.exp_slot_stride[1] : a.c.exp_slot_stride[0];
        Place<kFill> base_at;
        uint32_t used = 0, rounds = 0;  // a stage's bit: filled by this warp; parity of the last fill
        Walk<R> walk(a, start);
        Share sh{};
        int64_t units = start.u0;
        bool ok = true;
        for (; ok; ++item) {
            const Plan* g;
            if (kv == 0) {
                Segment seg;
                const bool any = walk.next(&seg);
                Plan p{};
                if (any) {
                    p = plan_of<PAIR>(a, seg);
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
            } else if ((g = plan_at(item)) == nullptr) {
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
            auto good = [&](int32_t page) { return page >= 0 && page < a.c.num_pages; };
            auto slot_of = [&](int k) { return (k * kTile + lane * 4 + in_page0) & (P - 1); };
            struct Exps {
                uint32_t e[4];
            };
            auto exps_of = [&](int k, int32_t page) {
                Exps x{};
                if (E4M3 && page != INT_MIN) {
                    const uint8_t* e = exps + exp_at(a.c, kv, good(page) ? page : 0, slot_of(k), h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x.e[i] = e[i * exp_step];
                }
                return x;
            };
            int32_t cur = entry(0), next = entry(1);
            Exps xc = exps_of(0, cur), xn = exps_of(1, next);
            Place<kFill> at = base_at;
            if (kv) at.advance(ring_v<PAIR>(0, n));
            for (int k = 0; k < n; ++k) {
                const int32_t after = entry(k + 2);
                const bool needed = cur != INT_MIN;
                // A page out of range: page 0 in its place, and NaN for the item.
                const bool bad = needed && !good(cur);
                if (at.round > 0 && !(ok = wait_all(&emptybar[at.stage], at.round - 1))) break;
                if (bad) {
                    cur = 0;
                    *reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) = 1;
                    if (a.status != nullptr) atomicOr(a.status + g->b, kBadPage);
                }
                if constexpr (E4M3) {
                    // Positions that no row sees may hold anything: factor 0, which
                    // the helpers turn into zeros. So do values that are NaN at
                    // positions that not every row sees; these are noted.
                    uint32_t top = 0, f[4], two = 0, hidden = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = k * kTile + lane * 4 + i;
                        if (p < any_lo || p > any_hi) {
                            hidden |= 1u << i;
                        } else if (xc.e[i] != 255u) {
                            top = max(top, xc.e[i]);
                        } else if (kv == 1 && (p < g->all_lo || p > g->all_hi)) {
                            hidden |= 1u << i;
                            const int x = atomicAdd(&ctl.noted[item % kItems], 1);
                            if (x < kNoted) ctl.note[item % kItems][x] = p;
                        }
                    }
                    top = __reduce_max_sync(0xFFFFFFFFu, top);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (kv == 0) {
                            f[i] = key_factor(xc.e[i], top);
                        } else {
                            const Factor x = factor_of(xc.e[i], T());
                            f[i] = x.f1;
                            two |= x.two && !(hidden >> i & 1u);
                        }
                        if (hidden >> i & 1u) f[i] = 0;
                    }
                    *reinterpret_cast<uint4*>(&ctl.factor[at.stage][lane * 4]) =
                        make_uint4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint32_t*>(&ctl.exps[at.stage][lane * 4]) =
                        xc.e[0] | xc.e[1] << 8 | xc.e[2] << 16 | xc.e[3] << 24;
                    const bool any_two = __any_sync(0xFFFFFFFFu, two != 0) != 0;
                    if (lane == 0) {
                        ctl.top[at.stage] = top;
                        ctl.two[at.stage] = any_two;
                    }
                    __syncwarp();
                }
                const bool leader = needed && first_of_box;
                const unsigned boxes = __ballot_sync(0xFFFFFFFFu, leader);
                if (lane == 0)
                    sv::mbar_arrive_expect_tx(&fullbar[at.stage], __popc(boxes) * box_bytes);
                __syncwarp();
                if (leader) {
                    const int c1 = slot_of(k);
                    if (E4M3) {
                        tma_load_4d(sr + at.stage * X::kRawBytes + lane_bytes, map, 0, c1, h, cur,
                                    &fullbar[at.stage]);
                    } else if (args.page_heads > 0) {
                        tma_load_5d(st + at.stage * X::kTileBytes + lane_bytes, map, 0, 0, 0, c1 >> 3,
                                    cur * args.page_heads + h * args.head_step, &fullbar[at.stage]);
                    } else {
#pragma unroll
                        for (int q = 0; q < DP / 64; ++q)
                            tma_load_4d(st + at.stage * X::kTileBytes + q * X::kPanel + lane_bytes,
                                        map, q * 64, c1, h, cur, &fullbar[at.stage]);
                    }
                }
                __syncwarp();
                used |= 1u << at.stage;
                rounds = (rounds & ~(1u << at.stage)) | (at.round & 1u) << at.stage;
                at.advance(kv ? ring_v_step<PAIR>(k, n) : ring_k_step<PAIR>(k));
                cur = next;
                next = after;
                xc = xn;
                xn = exps_of(k + 2, next);
            }
            base_at.advance(2 * n);
        }
        if (kv == 0 && lane == 0) {
            sh.units = start.U;
            args.shares[blockIdx.x] = sh;
        }
        if (!ok) {
            // No copy may be under way when the block ends.
            for (int i = 0; i < kFill; ++i)
                if (used >> i & 1u) sv::mbar_wait_bounded(&fullbar[i], rounds >> i & 1u, nullptr);
        }
    } else {
        // ------------------------------------------------------------------
        // Helpers: hidden values, and e4m3.
        // ------------------------------------------------------------------
        const int tid = (warp - 12) * 32 + lane;
        constexpr int kThreadsH = X::kHelpers * 32;
        Place<S> at;
        Place<kFill> raw_at;
        int k_tiles = 0;  // key tiles so far
        bool ok = true;
        for (; ok; ++item) {
            const Plan* g = plan_at(item);
            if (g == nullptr) break;
            const int n = g->n, inner_lo = g->inner_lo, inner_hi = g->inner_hi;
            auto note = [&](int p) {
                const int i = atomicAdd(&ctl.noted[item % kItems], 1);
                if (i < kNoted) ctl.note[item % kItems][i] = p;
            };
            int kk = 0, vv = 0;
            for (int i = 0; ok && i < 2 * n; ++i) {
                const bool is_v = vv < n && ring_v<PAIR>(vv, n) == i;
                const int k = is_v ? vv++ : kk++;
                const bool edge = !E4M3 && is_v && (k < inner_lo || k > inner_hi);
                if constexpr (!E4M3) {
                    if (!(ok = wait_all(&ctl.full[at.stage], at.round))) break;
                    if (edge) {
                        const uint32_t v = st + at.stage * X::kTileBytes;
                        constexpr int kLanes = DP / 8;  // lanes to a row
#pragma unroll 4
                        for (int x = tid; x < kTile * kLanes; x += kThreadsH) {
                            const int row = x / kLanes, ch = x % kLanes, p = k * kTile + row;
                            const uint32_t addr = v + tile_chunk(row, ch, args.group, args.panel);
                            const bool outside = p < g->any_lo || p > g->any_hi;
                            const bool common = p >= g->all_lo && p <= g->all_hi;
                            bool special = false;
                            if (!outside && !common)
                                special = any_special(ld_shared_v4(addr), exponent_mask(T()));
                            const unsigned m = __ballot_sync(0xFFFFFFFFu, special) >>
                                               (lane & ~(kLanes - 1));
                            const bool clear = (m & ((1ull << kLanes) - 1)) != 0;
                            if (outside || clear) st_shared_v4(addr, make_uint4(0, 0, 0, 0));
                            if (clear && ch == 0) note(p);
                        }
                        fence_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (edge) sv::mbar_arrive(&ctl.fixed[at.stage]);
                        sv::mbar_arrive(&ctl.empty[at.stage]);
                    }
                } else {
                    if (!(ok = wait_all(&ctl.raw_full[raw_at.stage], raw_at.round))) break;
                    if (at.round > 0 && !(ok = wait_all(&ctl.empty[at.stage], at.round - 1))) break;
                    const uint32_t raw = sr + raw_at.stage * X::kRawBytes;
                    const uint32_t dst = st + at.stage * X::kTileBytes;
                    // A thread expands 16 codes of a row, the same piece of every
                    // kStep-th row, two at a time. Eight neighbouring lanes take half of the
                    // pieces of two rows, the other half of the second: their
                    // 16-byte columns differ in the loads and, swizzled, in the
                    // stores.
                    constexpr int kPieces = DP / 16, kStep = kThreadsH / kPieces;
                    const int pair = tid / (2 * kPieces), odd = (tid >> 2) & 1;
                    const int row0 = pair * 2 + odd;
                    const int piece = (tid & 3) + (kPieces > 4 ? (((tid >> 3) & 1) ^ odd) << 2 : 0);
                    const bool in_row = piece * 16 < a.c.D;
                    const uint32_t from = raw + row0 * a.c.D + (in_row ? piece * 16 : 0);
                    const uint32_t to = dst + tile_chunk(row0, piece * 2, 1024, X::kPanel);
                    const uint32_t* factor = &ctl.factor[raw_at.stage][row0];
                    if (!is_v && tid == 0) ctl.k_scale[k_tiles & 3] = exp_value(ctl.top[raw_at.stage]);
                    constexpr int kBatch = 2;
                    auto expand_rows = [&](auto type) {
                        using U = decltype(type);
#pragma unroll 1
                        for (int r = 0; r < kTile; r += kBatch * kStep) {
                            uint4 codes[kBatch];
                            uint32_t f[kBatch];
#pragma unroll
                            for (int u = 0; u < kBatch; ++u) {
                                const int row = r + u * kStep;
                                codes[u] = ld_shared_v4(from + row * a.c.D);
                                f[u] = in_row ? factor[row] : 0u;
                            }
#pragma unroll
                            for (int u = 0; u < kBatch; ++u) {
                                // (a factor of zero: whatever the codes are)
                                if (f[u] == 0u) codes[u] = make_uint4(0, 0, 0, 0);
                                uint32_t o[8];
                                expand<U>(codes[u], f[u], o);
                                // (chunk 2 c + 1 is chunk 2 c's neighbour under the swizzle too)
                                const uint32_t t = to + (r + u * kStep) * 128;
                                st_shared_v4(t, make_uint4(o[0], o[1], o[2], o[3]));
                                st_shared_v4(t ^ 16u, make_uint4(o[4], o[5], o[6], o[7]));
                            }
                        }
                    };
                    if (is_v) {
                        expand_rows(T());
                        if (ctl.two[raw_at.stage] != 0) {
                            // Rare: some rows' second factor.
#pragma unroll 1
                            for (int r = 0; r < 2 * kTile; r += kStep) {
                                const uint32_t t = (to + (r >> 1) / kStep * kStep * 128) ^ ((r / kStep & 1) << 4);
                                const uint32_t f2 =
                                    factor_of(ctl.exps[raw_at.stage][row0 + (r >> 1) / kStep * kStep], T()).f2;
                                uint4 x = ld_shared_v4(t);
                                x = make_uint4(mul2(x.x, f2, T()), mul2(x.y, f2, T()),
                                               mul2(x.z, f2, T()), mul2(x.w, f2, T()));
                                st_shared_v4(t, x);
                            }
                        }
                    } else {
                        expand_rows(F16());
                    }
                    if (!is_v) ++k_tiles;
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        sv::mbar_arrive(&ctl.full[at.stage]);
                        sv::mbar_arrive(&ctl.raw_empty[raw_at.stage]);
                    }
                    raw_at.advance(1);
                }
                at.advance(1);
            }
        }
    }
    }
    __syncthreads();
    if (threadIdx.x == 0) args.shares[blockIdx.x].failed = *stop;
    if (warp == 8) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
}

// Joins the items that several blocks worked on, in block order: block x takes
// the item that block x of the tile kernel began and did not finish, a warp a
// row.
template <class T, int DP>
__global__ void __launch_bounds__(128) join_kernel(const Tiles args, int blocks)
{
    const Attn& a = args.a;
    const int lane = threadIdx.x & 31;
    sv::pdl_wait();
    const Share sh = args.shares[blockIdx.x];
    const float nan = __uint_as_float(0x7FFFFFFFu);
    if (sh.failed) {
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
    if (!sh.leads) return;
    const int r = blockIdx.y * (blockDim.x / 32) + (threadIdx.x >> 5);
    if (r >= sh.rows) return;
    constexpr int kPer = DP / 32;
    float m = __uint_as_float(sv::kF32NegInfBits), l = 0.f, o[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = 0.f;
    for (int c = blockIdx.x; c <= sh.last; ++c) {
        if (share_begin(sh.units, c, blocks) == share_begin(sh.units, c + 1, blocks)) continue;
        const float* p = args.part +
                         ((static_cast<int64_t>(c) * 2 + (c == static_cast<int>(blockIdx.x) ? 1 : 0)) *
                              args.part_rows + r) * (DP + 4);
        const float pm = p[DP], pl = p[DP + 1];
        const float mn = fmaxf(m, pm);
        const float keep = m == mn ? 1.f : sv::ex2(m - mn);
        const float w = pm == mn ? 1.f : sv::ex2(pm - mn);
        l = l * keep + pl * w;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + p[lane + 32 * i] * w;
        m = mn;
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
bool make_map(CUtensorMap* map, const Cache& c, int kv, bool f16, bool e4m3)
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
              e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// 16-bit rows of 128 elements, one copy a page for both halves of the rows:
// [page and head][slot / 8][half][slot % 8][64 elements]. Pages and heads are one
// axis, in steps of a head (one head: of a page); see heads_to_a_page.
bool make_map5(CUtensorMap* map, const Cache& c, int kv, bool f16, int64_t page_heads)
{
    const EncodeTiled fn = encode_fn();
    if (fn == nullptr) return false;
    const int P = 1 << c.page_shift;
    const int64_t step = c.Hkv > 1 ? c.head_stride[kv] : c.page_stride[kv];
    const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(P / 8),
                                static_cast<cuuint64_t>((c.num_pages - 1) * page_heads + c.Hkv)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(c.slot_stride[kv]), 128,
                                   static_cast<cuuint64_t>(c.slot_stride[kv]) * 8,
                                   static_cast<cuuint64_t>(step)};
    const cuuint32_t box[5] = {64, 8, 2, static_cast<cuuint32_t>((P < kTile ? P : kTile) / 8), 1};
    const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
    return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
              c.pages[kv], dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How far apart pages are on make_map5's axis of pages and heads; 0 where it
// cannot be used: the page stride has to be a multiple of the head stride, the
// same in keys and values.
int64_t heads_to_a_page(const Cache& c, bool e4m3)
{
    if (e4m3 || c.D != 128) return 0;
    int64_t n = 1;
    if (c.Hkv > 1) {
        if (c.head_stride[0] <= 0 || c.page_stride[0] % c.head_stride[0] != 0) return 0;
        n = c.page_stride[0] / c.head_stride[0];
        if (n <= 0 || c.head_stride[1] <= 0 || c.page_stride[1] != n * c.head_stride[1]) return 0;
    }
    // (coordinates are 32 bits)
    return n < (int64_t(1) << 31) / c.num_pages - c.Hkv ? n : 0;
}

template <class T, int DP, bool E4M3, bool PAIR>
cudaError_t launch_shape(const CUtensorMap& k, const CUtensorMap& v, const Tiles& t, int blocks,
                         int64_t rows, cudaStream_t s)
{
    using X = Shape<DP, E4M3, PAIR>;
    using Ctl = Control<X::kStages, X::kRawStages, PAIR>;
    constexpr size_t smem = X::kTiles + sizeof(Ctl);
    static_assert(smem <= kMaxSmem, "shared memory");
    // (factor is written 16 bytes at a time)
    static_assert(alignof(Ctl) == 16 && X::kTiles % 1024 == 0, "alignment");
    auto* f = tiles_kernel<T, DP, E4M3, PAIR>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (E4M3) {
        // (the split of registers waits for what the block was not launched with)
        static const int regs = [f] {
            cudaFuncAttributes at{};
            return cudaFuncGetAttributes(&at, f) == cudaSuccess ? at.numRegs : 0;
        }();
        if (regs < X::kRegsLaunch) return cudaErrorInvalidConfiguration;
    }
    f<<<blocks, X::kThreads, smem, s>>>(k, v, t);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
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

template <class T, int DP>
cudaError_t launch_type(const CUtensorMap& k, const CUtensorMap& v, const Tiles& t, int blocks,
                        int64_t rows, bool e4m3, bool pair, cudaStream_t s)
{
    if (e4m3)
        return pair ? launch_shape<T, DP, true, true>(k, v, t, blocks, rows, s)
                    : launch_shape<T, DP, true, false>(k, v, t, blocks, rows, s);
    return pair ? launch_shape<T, DP, false, true>(k, v, t, blocks, rows, s)
                : launch_shape<T, DP, false, false>(k, v, t, blocks, rows, s);
}

// Rows of the largest item.
int64_t item_rows(int64_t max_chunk, int64_t G) { return max_chunk * G < 256 ? max_chunk * G : 256; }

constexpr size_t kShareBytes = (sizeof(Share) * kMaxBlocks + 255) / 256 * 256;

}  // namespace

size_t tiles_workspace(int64_t max_chunk, int64_t G, int64_t D)
{
    const int64_t dp = D <= 64 ? 64 : 128;
    return kShareBytes + static_cast<size_t>(kMaxBlocks) * 2 * item_rows(max_chunk, G) * (dp + 4) *
                             sizeof(float);
}

cudaError_t launch_attention_tiles(const Attn& a, bool f16, bool e4m3, void* workspace,
                                   cudaStream_t s, bool* mapped)
{
    CUtensorMap k, v;
    const int64_t page_heads = heads_to_a_page(a.c, e4m3);
    const bool five = page_heads > 0 && make_map5(&k, a.c, 0, f16, page_heads) &&
                      make_map5(&v, a.c, 1, f16, page_heads);
    *mapped = five || (make_map(&k, a.c, 0, f16, e4m3) && make_map(&v, a.c, 1, f16, e4m3));
    if (!*mapped) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    const int64_t rows = item_rows(a.max_chunk, a.G);
    Tiles t{a, reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kShareBytes),
            static_cast<Share*>(workspace), static_cast<int32_t>(rows),
            five ? 2048 : 1024, five ? 1024 : kTile * 128,
            five ? static_cast<int32_t>(page_heads) : 0, a.c.Hkv > 1 ? 1 : 0};
    const bool pair = rows > 128;
    if (a.c.D <= 64)
        return f16 ? launch_type<F16, 64>(k, v, t, blocks, rows, e4m3, pair, s)
                   : launch_type<Bf16, 64>(k, v, t, blocks, rows, e4m3, pair, s);
    return f16 ? launch_type<F16, 128>(k, v, t, blocks, rows, e4m3, pair, s)
               : launch_type<Bf16, 128>(k, v, t, blocks, rows, e4m3, pair, s);
}

}  // namespace sva
