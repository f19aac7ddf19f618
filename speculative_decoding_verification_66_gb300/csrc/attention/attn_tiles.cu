// attn_tiles.cu -- attention over the paged cache on the 5th-generation tensor
// cores, head sizes up to 128.
//
// For a block of query rows Q and the keys K and values V of a 128-key tile
//   S = Q K^T,  m' = max(m, max S),  P = 2^(c S - m'),
//   l' = l 2^(m - m') + sum P,  O' = O 2^(m - m') + P V,
// with c = scale log2(e): one pass over the cache, the softmax never leaves the
// chip. S, P and O live in tensor memory, a row to a lane: a thread owns a row,
// so the maximum and the sum need no exchange between threads. O is rescaled
// only when the maximum has grown by more than 2^kSlack since the last time
// (the weights stay below 2^kSlack; the sum is exact either way), which is
// rare after the first tiles.
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
//   8         issues the products
//   9         loads: page numbers, one bulk tensor copy a page and 64 elements,
//             exponents
//   10-..     16-bit caches: makes the values at a tile's hidden positions
//             harmless. e4m3 caches: also expand every tile to the query's
//             type, exactly (see e4m3_words), into the stage that the products
//             read.
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
// Work is shared among one block per SM as attn_plan.cuh says; items that
// several blocks share are joined by join_kernel in block order, so results
// depend on the lengths and the number of blocks alone.
#include <climits>

#include "attn_internal.h"
#include "attn_plan.cuh"
#include "tensor_core.cuh"

namespace sva {
namespace {

constexpr float kSlack = 8.f;
constexpr int kMaxBlocks = 160;  // shares in the workspace; grids are no larger
constexpr int kNoted = 8;        // noted positions an item can hold
constexpr int kItems = 8;        // items whose notes are kept at one time
constexpr size_t kMaxSmem = 232448;

template <int DP, bool E4M3, bool PAIR>
struct Shape {
    static constexpr int kRows = PAIR ? 256 : 128;
    static constexpr int kTileBytes = kTile * DP * 2;  // a K or V tile as the products read it
    static constexpr int kRawBytes = E4M3 ? kTile * DP : 0;
    static constexpr int kQBytes = kRows * DP * 2;
    // Stages in tiles of K or V: what the SM's shared memory holds. (The loads
    // and the notes of hidden values run at most kStages + kRawStages tiles, half
    // as many items, ahead of the products: below kItems.)
    static constexpr int kStages = DP == 128 ? (E4M3 ? 3 : (PAIR ? 5 : 6)) : (E4M3 ? 4 : 8);
    static constexpr int kRawStages = E4M3 ? (DP == 128 ? (PAIR ? 4 : 5) : 8) : 0;
    static_assert((kStages + kRawStages) / 2 < kItems - 1, "notes");
    static constexpr int kHelpers = E4M3 ? 8 : 4;
    static constexpr int kThreads = (10 + kHelpers) * 32;
    static constexpr int kPanel = kTile * 128;  // bytes of 64 elements of every row
    static constexpr int kTiles = kQBytes + kStages * kTileBytes + kRawStages * kRawBytes;
};

// Shared memory besides the tiles.
template <int STAGES, int RAW, bool PAIR>
struct Control {
    uint64_t full[STAGES], empty[STAGES], fixed[STAGES];
    uint64_t raw_full[RAW > 0 ? RAW : 1], raw_empty[RAW > 0 ? RAW : 1];
    uint64_t s_full[2], p_ready[2], q_ready, o_full, ml_ready, done;
    uint32_t tmem;
    int stop;
    Start start;
    int64_t sums[18];
    int noted[kItems];             // how many positions are noted
    uint32_t note[kItems][kNoted]; // which
    int bad_page[kItems];
    float2 ml[2][PAIR ? 1 : kTile]; // a row's maximum and sum in either slot
    uint8_t exps[RAW > 0 ? RAW : 1][kTile];
};

struct Tiles {
    Attn a;
    float* part;   // [blocks][2][rows][part_cols]: unnormalised O, then m and l
    Share* shares; // [blocks]
    int32_t part_rows;
};

// Where the tiles of a segment lie in the ring: the order in which the products
// use them. PAIR: K0 V0 K1 V1 ..; otherwise K0 K1 V0 K2 V1 .., since the second
// slot's scores come before the first slot's values.
template <bool PAIR>
__device__ __forceinline__ int64_t ring_k(int64_t base, int k)
{
    return base + (PAIR ? 2 * k : (k == 0 ? 0 : 2 * k - 1));
}
template <bool PAIR>
__device__ __forceinline__ int64_t ring_v(int64_t base, int k, int n)
{
    return base + (PAIR ? 2 * k + 1 : (k == n - 1 ? 2 * k + 1 : 2 * k + 2));
}

// The tiles of a segment that slot s works on: [lo, hi) in steps of `step`.
struct SlotTiles {
    int lo, hi, step;
};
template <bool PAIR>
__device__ __forceinline__ SlotTiles slot_tiles(const Attn& a, const Segment& g, int s)
{
    if (!PAIR) return SlotTiles{g.t.lo + s, g.t.hi, 2};
    const int r0 = g.row0 + 128 * s, r1 = min(g.row0 + g.rows, r0 + 128);
    if (r0 >= r1) return SlotTiles{g.t.hi, g.t.hi, 1};
    const Range t = row_tiles(a, g.cached, r0, r1);
    return SlotTiles{max(g.t.lo, t.lo), min(g.t.hi, t.hi), 1};
}
__device__ __forceinline__ bool works_on(const SlotTiles& t, int j)
{
    return j >= t.lo && j < t.hi && (t.step == 1 || ((j - t.lo) & 1) == 0);
}

// The positions that every row of an item sees, and those that any row sees,
// relative to tile j: [lo, hi] each. Beyond `all` a tile needs its hidden
// values made harmless.
struct Seen {
    int64_t all_lo, all_hi, any_lo, any_hi;
};
__device__ __forceinline__ Seen item_seen(const Attn& a, const Segment& g)
{
    const int64_t p0 = g.cached + g.row0 / a.G, p1 = g.cached + (g.row0 + g.rows - 1) / a.G;
    return Seen{first_key(a, p1), p0, first_key(a, p0), p1};
}
__device__ __forceinline__ bool at_edge(const Seen& s, int j)
{
    const int64_t lo = static_cast<int64_t>(j) << kTileShift;
    return lo < s.all_lo || lo + kTile - 1 > s.all_hi;
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
    if (e == 255u) return Factor{both(0x7FFFu), both(0x3F80u), false};
    const uint32_t x = min(e, 134u), y = e - x;
    return Factor{both((x + 120u) << 7), both((y + 127u) << 7), y != 0};
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
template <class T>
__device__ __forceinline__ void e4m3_words(uint4 codes, const Factor& f, uint4* lo, uint4* hi)
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint2 s = spread(w[i], T());
        o[2 * i] = mul2(s.x, f.f1, T());
        o[2 * i + 1] = mul2(s.y, f.f1, T());
    }
    if (f.two) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = mul2(o[i], f.f2, T());
    }
    *lo = make_uint4(o[0], o[1], o[2], o[3]);
    *hi = make_uint4(o[4], o[5], o[6], o[7]);
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
// Byte offset of 16-byte chunk `chunk` of a row in a tile of 64-element panels
// with the 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_chunk(int row, int chunk, int panel_bytes)
{
    return (chunk >> 3) * panel_bytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// Scores at columns [0, lo) and (hi, 127] of a tile do not count.
struct Columns {
    int lo, hi;
};

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
            // (16-bit: the helpers, too, pass every tile in order, or a parity
            // would stand for another round of the stage than they mean)
            sv::mbar_init(&ctl.empty[i], E4M3 ? 1 : 1 + X::kHelpers);
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
        sv::mbar_init(&ctl.o_full, 1);
        sv::mbar_init(&ctl.ml_ready, 8);
        sv::mbar_init(&ctl.done, 1);
        // (The swizzle needs tiles on 1024-byte boundaries. There is no static
        // shared memory before them, so they are; if not, the call fails.)
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
    Walk<R> walk(a, start);
    Segment g;
    int item = 0;  // segments taken so far

    if (warp < 8) {
        // ------------------------------------------------------------------
        // Softmax of slot s; thread = row.
        // ------------------------------------------------------------------
        const int s = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t s_addr = lane_base + s * 128, o_addr = lane_base + 256 + s * DP;
        const float c = a.scale_log2;
        const float ninf = __uint_as_float(sv::kF32NegInfBits);
        uint32_t tiles_done = 0;
        bool ok = true;
        for (; ok && walk.next(&g); ++item) {
            // The queries: rows of 64-element panels, swizzled; zeros past D.
            {
                constexpr int kChunks = DP / 8;
                const int first = PAIR ? s * 128 : s * 64, count = PAIR ? 128 : 64;
                const int tid = threadIdx.x & 127;
#pragma unroll 4
                for (int i = tid; i < count * kChunks; i += 128) {
                    const int r = first + i / kChunks, ch = i % kChunks;
                    if (r >= g.rows) continue;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    const int rr = g.row0 + r, t = rr / a.G;
                    if (ch * 8 < a.c.D)
                        v = *reinterpret_cast<const uint4*>(
                            a.q + (static_cast<int64_t>(g.q0) + t) * a.q_token +
                            static_cast<int64_t>(g.h * a.G + (rr - t * a.G)) * a.q_head + ch * 16);
                    st_shared_v4(sq + (PAIR ? s * 128 * DP * 2 : 0) +
                                     tile_chunk(PAIR ? r - first : r, ch, X::kPanel),
                                 v);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.q_ready);
            }
            const int slot_row = PAIR ? 128 * s + row : row;  // row of the item
            const int warp_row = PAIR ? 128 * s + quad * 32 : quad * 32;
            const bool live = warp_row < g.rows;  // some row of this warp exists
            const int r = g.row0 + min(slot_row, g.rows - 1);
            const int64_t pos = g.cached + r / a.G;  // last position seen
            const int64_t low = first_key(a, pos);
            const SlotTiles mine = slot_tiles<PAIR>(a, g, s);
            float m = ninf, l = 0.f;
            bool begun = false;
            for (int j = mine.lo; j < mine.hi; j += mine.step) {
                if (!(ok = wait_all(&ctl.s_full[s], tiles_done))) break;
                ++tiles_done;
                if (live) {
                    fence_after();
                    const int64_t p0 = static_cast<int64_t>(j) << kTileShift;
                    const int clo = static_cast<int>(max(low - p0, int64_t(0)));
                    const int chi = static_cast<int>(min(pos - p0, int64_t(kTile - 1)));
                    const bool masked =
                        __any_sync(0xFFFFFFFFu, clo > 0 || chi < kTile - 1) != 0;
                    float top = ninf;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float v[32];
                        tmem_ld32(s_addr + 32 * k, v);
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = 32 * k + i >= clo && 32 * k + i <= chi ? v[i] : ninf;
                        }
                        float t0 = v[0], t1 = v[1];
#pragma unroll
                        for (int i = 2; i < 32; i += 2) {
                            t0 = fmaxf(t0, v[i]);
                            t1 = fmaxf(t1, v[i + 1]);
                        }
                        top = fmaxf(top, fmaxf(t0, t1));
                    }
                    const float mt = top * c;  // (scale > 0)
                    const bool grow = mt > m + kSlack || (!begun && mt > m);
                    if (begun && __any_sync(0xFFFFFFFFu, grow)) {
                        // The slot's products so far are complete: s_full's commit
                        // came after them.
                        const float keep = grow ? sv::ex2(m - mt) : 1.f;
#pragma unroll 1
                        for (int k = 0; k < DP / 32; ++k) {
                            float v[32];
                            tmem_ld32(o_addr + 32 * k, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= keep;
                            tmem_st32(o_addr + 32 * k, v);
                        }
                        l *= keep;
                    }
                    if (grow) m = mt;
                    begun = true;
                    const float shift = m == ninf ? 0.f : -m;
                    float l0 = 0.f, l1 = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float v[32];
                        uint32_t w[16];
                        tmem_ld32(s_addr + 32 * k, v);
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = 32 * k + i >= clo && 32 * k + i <= chi ? v[i] : ninf;
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float p0f = sv::ex2(fmaf(v[i], c, shift));
                            const float p1f = sv::ex2(fmaf(v[i + 1], c, shift));
                            l0 += p0f;
                            l1 += p1f;
                            w[i / 2] = narrow2(p0f, p1f, T());
                        }
                        tmem_st16(s_addr + 16 * k, w);
                    }
                    l += l0 + l1;
                    tmem_wait_st();
                    fence_before();
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.p_ready[s]);
            }
            if (!ok) break;

            // --------------------------------------------------------------
            // The rows' results.
            // --------------------------------------------------------------
            bool has[2] = {begun, false};
            float wt[2] = {1.f, 0.f};
            if (!PAIR) {
                ctl.ml[s][row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.ml_ready);
                if (!(ok = wait_all(&ctl.ml_ready, item))) break;
                const float2 x0 = ctl.ml[0][row], x1 = ctl.ml[1][row];
                has[0] = g.t.lo < g.t.hi;
                has[1] = g.t.lo + 1 < g.t.hi;
                m = fmaxf(x0.x, x1.x);
                wt[0] = x0.x == m ? 1.f : sv::ex2(x0.x - m);
                wt[1] = x1.x == m ? 1.f : sv::ex2(x1.x - m);
                l = x0.y * wt[0] + x1.y * wt[1];
            }
            if (!(ok = wait_all(&ctl.o_full, item))) break;
            fence_after();
            const bool whole = g.t.lo == g.item.lo && g.t.hi == g.item.hi;
            const bool valid = slot_row < g.rows;
            // A row that sees a noted position is computed again below.
            const int noted = *reinterpret_cast<volatile int*>(&ctl.noted[item % kItems]);
            const bool bad = *reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) != 0;
            bool again = noted > kNoted;
            for (int i = 0; i < min(noted, kNoted); ++i) {
                const int64_t p = *reinterpret_cast<volatile uint32_t*>(&ctl.note[item % kItems][i]);
                again |= p >= low && p <= pos;
            }
            again = again && valid && !bad;
            const float nan = __uint_as_float(0x7FFFFFFFu);
            const float inv = bad ? nan : (whole ? 1.f / l : 1.f);
            const int64_t orow = valid ? out_row(a, g.q0, g.h, r) : 0;
            float* part = args.part +
                          ((static_cast<int64_t>(blockIdx.x) * 2 + (g.t.lo == g.item.lo ? 1 : 0)) *
                               args.part_rows + slot_row) * (DP + 4);
            if (live) {
                // !PAIR: slot s writes its half of the columns.
                constexpr int kParts = DP / 32;
                const int k0 = PAIR ? 0 : s * kParts / 2, k1 = PAIR ? kParts : (s + 1) * kParts / 2;
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                    float o[32];
                    __syncwarp();
                    if (PAIR) {
                        if (has[0]) {
                            tmem_ld32(o_addr + 32 * k, o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0.f;
                        }
                    } else {
                        tmem_ld32(lane_base + 256 + 32 * k, o);
                        if (has[1]) {
                            float p[32];
                            tmem_ld32(lane_base + 256 + DP + 32 * k, p);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = o[i] * wt[0] + p[i] * wt[1];
                        }
                    }
                    if (!valid || again) continue;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            if (32 * k + i < a.c.D)
                                *reinterpret_cast<uint4*>(a.out +
                                                          (orow * a.c.D + 32 * k + i) * 2) =
                                    make_uint4(narrow2(o[i] * inv, o[i + 1] * inv, T()),
                                               narrow2(o[i + 2] * inv, o[i + 3] * inv, T()),
                                               narrow2(o[i + 4] * inv, o[i + 5] * inv, T()),
                                               narrow2(o[i + 6] * inv, o[i + 7] * inv, T()));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(part + 32 * k + i) =
                                make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
                    }
                }
                __syncwarp();
                if (valid && !again && (PAIR || s == 0)) {
                    if (!whole) {
                        part[DP] = m;
                        part[DP + 1] = bad ? nan : l;
                    } else if (a.lse != nullptr) {
                        a.lse[orow] = bad ? nan : fmaf(m, kLn2, logf(l));
                    }
                }
                unsigned todo = PAIR || s == 0 ? __ballot_sync(0xFFFFFFFFu, again) : 0u;
                while (todo != 0) {
                    const int i = __ffs(static_cast<int>(todo)) - 1;
                    todo &= todo - 1;
                    const int ri = g.row0 + warp_row + i;
                    const int64_t pi = g.cached + ri / a.G, row_i = out_row(a, g.q0, g.h, ri);
                    const int64_t lo = max(first_key(a, pi), static_cast<int64_t>(g.t.lo) << kTileShift);
                    const int64_t hi = min(pi + 1, static_cast<int64_t>(g.t.hi) << kTileShift);
                    const int64_t t = row_i / a.Hq;
                    float om, ol, o[8];
                    attend_row<T, E4M3>(a, g.b, g.h, a.q + t * a.q_token + (row_i - t * a.Hq) * a.q_head,
                                        lo, hi, lane, &om, &ol, o);
                    if (whole) {
                        const float x = 1.f / ol;
                        if (lane * 8 < a.c.D)
                            *reinterpret_cast<uint4*>(a.out + (row_i * a.c.D + lane * 8) * 2) =
                                make_uint4(narrow2(o[0] * x, o[1] * x, T()),
                                           narrow2(o[2] * x, o[3] * x, T()),
                                           narrow2(o[4] * x, o[5] * x, T()),
                                           narrow2(o[6] * x, o[7] * x, T()));
                        if (a.lse != nullptr && lane == 0) a.lse[row_i] = fmaf(om, kLn2, logf(ol));
                    } else {
                        float* p = args.part +
                                   ((static_cast<int64_t>(blockIdx.x) * 2 +
                                     (g.t.lo == g.item.lo ? 1 : 0)) * args.part_rows +
                                    warp_row + i) * (DP + 4);
                        if (lane * 8 < DP) {
                            *reinterpret_cast<float4*>(p + lane * 8) =
                                make_float4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<float4*>(p + lane * 8 + 4) =
                                make_float4(o[4], o[5], o[6], o[7]);
                        }
                        if (lane == 0) {
                            p[DP] = om;
                            p[DP + 1] = ol;
                        }
                    }
                }
                fence_before();
            }
            // The notes of the item before: every warp has read them (this item's
            // products began after all had), and the item that gets their place
            // waits for products that come after this thread's next arrival.
            __syncwarp();
            if (threadIdx.x == 0) {
                ctl.noted[(item + kItems - 1) % kItems] = 0;
                ctl.bad_page[(item + kItems - 1) % kItems] = 0;
            }
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------------
        // Products, from one lane.
        // ------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t id_s = idesc<T, kTile, false>(), id_o = idesc<T, DP, true>();
            int64_t ring = 0;
            uint32_t fixes = 0;      // parity of each stage's next fix
            uint32_t p_count[2] = {0, 0};
            bool ok = true;
            for (; ok && walk.next(&g); ++item) {
                if (!(ok = wait(&ctl.q_ready, item))) break;
                fence_after();
                const int n = g.t.hi - g.t.lo;
                const SlotTiles mine[2] = {slot_tiles<PAIR>(a, g, 0), slot_tiles<PAIR>(a, g, 1)};
                const Seen seen = item_seen(a, g);
                bool out[2] = {false, false}, begun[2] = {false, false};
                int qj = g.t.lo, qs = 0, vj = g.t.lo, vs = 0;
                auto settle = [&](int& j, int& s) {
                    while (j < g.t.hi && !works_on(mine[s], j)) {
                        s ^= 1;
                        if (s == 0) ++j;
                    }
                };
                auto last_user = [&](int j, int s) { return s == 1 || !works_on(mine[1], j); };
                settle(qj, qs);
                settle(vj, vs);
                while (vj < g.t.hi) {
                    while (qj < g.t.hi && !out[qs]) {
                        const int64_t at = ring_k<PAIR>(ring, qj - g.t.lo);
                        const int stage = static_cast<int>(at % S);
                        if (!(ok = wait(&ctl.full[stage], static_cast<uint32_t>(at / S)))) break;
                        fence_after();
                        const uint32_t q = sq + (PAIR ? qs * 128 * DP * 2 : 0);
                        const uint32_t k = st + stage * X::kTileBytes;
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) {
                            const uint32_t o = (i >> 2) * X::kPanel + (i & 3) * 32;
                            mma_ss(tmem + qs * 128, smem_desc(q + o, 16), smem_desc(k + o, 16), id_s,
                                   i > 0);
                        }
                        mma_commit(&ctl.s_full[qs]);
                        if (last_user(qj, qs)) mma_commit(&ctl.empty[stage]);
                        out[qs] = true;
                        qs ^= 1;
                        if (qs == 0) ++qj;
                        settle(qj, qs);
                    }
                    if (!ok) break;
                    const int64_t at = ring_v<PAIR>(ring, vj - g.t.lo, n);
                    const int stage = static_cast<int>(at % S);
                    if (!(ok = wait(&ctl.full[stage], static_cast<uint32_t>(at / S)))) break;
                    if (!E4M3 && at_edge(seen, vj) && (PAIR ? (vs == 0 || !works_on(mine[0], vj)) : true)) {
                        if (!(ok = wait(&ctl.fixed[stage], fixes >> stage))) break;
                        fixes ^= 1u << stage;
                    }
                    if (!(ok = wait(&ctl.p_ready[vs], p_count[vs]))) break;
                    ++p_count[vs];
                    fence_after();
                    const uint32_t v = st + stage * X::kTileBytes;
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i)
                        mma_ts(tmem + 256 + vs * DP, tmem + vs * 128 + i * 8,
                               smem_desc(v + i * 2048, X::kPanel), id_o, begun[vs] || i > 0);
                    begun[vs] = true;
                    out[vs] = false;
                    if (last_user(vj, vs)) mma_commit(&ctl.empty[stage]);
                    vs ^= 1;
                    if (vs == 0) ++vj;
                    settle(vj, vs);
                }
                if (!ok) break;
                mma_commit(&ctl.o_full);
                ring += 2 * n;
            }
            // Everything issued has completed once this arrives.
            mma_commit(&ctl.done);
            sv::mbar_wait_bounded(&ctl.done, 0, nullptr);
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------------
        // Copies.
        // ------------------------------------------------------------------
        uint64_t* fullbar = E4M3 ? ctl.raw_full : ctl.full;
        uint64_t* emptybar = E4M3 ? ctl.raw_empty : ctl.empty;
        const int P = 1 << a.c.page_shift, box = min(P, kTile);
        const int row_bytes = a.c.D;  // of a raw e4m3 row
        int64_t ring = 0, issued = 0;
        bool ok = true;
        for (; ok && walk.next(&g); ++item) {
            const int n = g.t.hi - g.t.lo;
            const Seen seen = item_seen(a, g);
            // Page and exponents of this lane's four positions in tile k; loaded
            // one tile ahead.
            auto page_at = [&](int k) {
                const int64_t p = (static_cast<int64_t>(g.t.lo + k) << kTileShift) + lane * 4;
                // (a page is needed if any of its positions is seen)
                const int64_t page0 = p & ~static_cast<int64_t>(P - 1);
                if (k >= n || page0 > seen.any_hi || page0 + P - 1 < seen.any_lo) return INT_MIN;
                return page_of(a.c, g.b, p);
            };
            auto load_tile = [&](int kv, int k, int32_t page) {
                const int64_t at = kv == 0 ? ring_k<PAIR>(ring, k) : ring_v<PAIR>(ring, k, n);
                const int stage = static_cast<int>(at % kFill);
                const int64_t round = at / kFill;
                const bool needed = page != INT_MIN;
                // A page out of range: page 0 in its place, and NaN for the item.
                const bool bad = needed && page < 0;
                if (bad) page = 0;
                const int slot = (lane * 4) & (P - 1);
                const int64_t p = (static_cast<int64_t>(g.t.lo + k) << kTileShift) + lane * 4;
                uint32_t e4 = 0;
                if (E4M3 && needed) {
                    const uint8_t* e = (kv ? a.c.exps[1] : a.c.exps[0]) +
                                       exp_at(a.c, kv, page, static_cast<int32_t>(p) & (P - 1), g.h);
                    const int64_t es = kv ? a.c.exp_slot_stride[1] : a.c.exp_slot_stride[0];
#pragma unroll
                    for (int i = 0; i < 4; ++i) e4 |= static_cast<uint32_t>(e[i * es]) << (8 * i);
                }
                if (round > 0 && !wait_all(&emptybar[stage], static_cast<uint32_t>(round - 1)))
                    return false;
                if (bad) {
                    *reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) = 1;
                    if (a.status != nullptr) atomicOr(a.status + g.b, kBadPage);
                }
                if (E4M3) *reinterpret_cast<uint32_t*>(&ctl.exps[stage][lane * 4]) = e4;
                // One lane a box: the lane whose first position is the box's first.
                const bool leader = needed && (P >= kTile ? lane == 0 : slot == 0);
                const unsigned boxes = __ballot_sync(0xFFFFFFFFu, leader);
                const uint32_t bytes = E4M3 ? box * row_bytes : box * DP * 2;
                __syncwarp();
                if (lane == 0)
                    sv::mbar_arrive_expect_tx(&fullbar[stage], __popc(boxes) * bytes);
                __syncwarp();
                if (leader) {
                    const CUtensorMap* map = kv ? &vmap : &kmap;
                    const int c1 = static_cast<int>(p) & (P - 1);
                    if (E4M3) {
                        tma_load_4d(sr + stage * X::kRawBytes + lane * 4 * row_bytes, map, 0, c1,
                                    g.h, page, &fullbar[stage]);
                    } else {
#pragma unroll
                        for (int q = 0; q < DP / 64; ++q)
                            tma_load_4d(st + stage * X::kTileBytes + q * X::kPanel + lane * 512,
                                        map, q * 64, c1, g.h, page, &fullbar[stage]);
                    }
                }
                issued = at + 1;
                return true;
            };
            int32_t cur = page_at(0), next = page_at(1);
            ok = load_tile(0, 0, cur);
            for (int k = 0; ok && k < n; ++k) {
                const int32_t after = page_at(k + 2);
                if (PAIR) {
                    ok = load_tile(1, k, cur) && (k + 1 >= n || load_tile(0, k + 1, next));
                } else {
                    ok = (k + 1 >= n || load_tile(0, k + 1, next)) && load_tile(1, k, cur);
                }
                cur = next;
                next = after;
            }
            ring += 2 * n;
        }
        if (!ok) {
            // No copy may be under way when the block ends.
            const int64_t first = issued > kFill ? issued - kFill : 0;
            for (int64_t i = first; i < issued; ++i)
                sv::mbar_wait_bounded(&fullbar[i % kFill], static_cast<uint32_t>((i / kFill) & 1),
                                      nullptr);
        }
    } else {
        // ------------------------------------------------------------------
        // Helpers: hidden values, and e4m3.
        // ------------------------------------------------------------------
        const int helper = warp - 10, tid = helper * 32 + lane;
        constexpr int kThreadsH = X::kHelpers * 32;
        int64_t ring = 0;
        bool ok = true;
        for (; ok && walk.next(&g); ++item) {
            const int n = g.t.hi - g.t.lo;
            const Seen seen = item_seen(a, g);
            auto note = [&](int64_t p) {
                const int i = atomicAdd(&ctl.noted[item % kItems], 1);
                if (i < kNoted) ctl.note[item % kItems][i] = static_cast<uint32_t>(p);
            };
            // Every tile in ring order.
            int kk = 0, vv = 0;
            for (int i = 0; ok && i < 2 * n; ++i) {
                const int64_t at = ring + i;
                const bool is_v = vv < n && ring_v<PAIR>(ring, vv, n) == at;
                const int j = g.t.lo + (is_v ? vv++ : kk++);
                const bool edge = is_v && at_edge(seen, j);
                const int64_t p0 = static_cast<int64_t>(j) << kTileShift;
                const int cs = static_cast<int>(at % S);
                if constexpr (!E4M3) {
                    if (!(ok = wait_all(&ctl.full[cs], static_cast<uint32_t>(at / S)))) break;
                    if (edge) {
                        const uint32_t v = st + cs * X::kTileBytes;
                        constexpr int kLanes = DP / 8;  // lanes to a row
#pragma unroll 4
                        for (int x = tid; x < kTile * kLanes; x += kThreadsH) {
                            const int row = x / kLanes, ch = x % kLanes;
                            const int64_t p = p0 + row;
                            const uint32_t addr = v + tile_chunk(row, ch, X::kPanel);
                            const bool outside = p < seen.any_lo || p > seen.any_hi;
                            const bool common = p >= seen.all_lo && p <= seen.all_hi;
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
                        if (edge) sv::mbar_arrive(&ctl.fixed[cs]);
                        sv::mbar_arrive(&ctl.empty[cs]);
                    }
                } else {
                    const int rs = static_cast<int>(at % RS);
                    if (!(ok = wait_all(&ctl.raw_full[rs], static_cast<uint32_t>(at / RS)))) break;
                    if (at >= S &&
                        !(ok = wait_all(&ctl.empty[cs], static_cast<uint32_t>(at / S - 1))))
                        break;
                    const uint32_t raw = sr + rs * X::kRawBytes, dst = st + cs * X::kTileBytes;
                    // A thread expands 16 codes of a row. Eight lanes of a phase
                    // of the stores take four pieces of two rows, whose swizzled
                    // 16-byte columns differ.
                    constexpr int kPieces = DP / 16;
#pragma unroll
                    for (int t = 0; t < kTile * kPieces / kThreadsH; ++t) {
                        const int x = t * kThreadsH + tid;
                        const int row = (x / (8 * kPieces / 4)) * 2 + ((x >> 2) & 1);
                        const int piece = (x & 3) + (((x >> 3) % (kPieces / 4)) << 2);
                        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                        const uint32_t e = ctl.exps[rs][row];
                        bool use = piece * 16 < a.c.D;
                        if (edge) {
                            const int64_t p = p0 + row;
                            const bool outside = p < seen.any_lo || p > seen.any_hi;
                            const bool common = p >= seen.all_lo && p <= seen.all_hi;
                            if (outside) use = false;
                            if (!outside && !common && e == 255u) {
                                use = false;
                                if (piece == 0) note(p);
                            }
                        }
                        if (use)
                            e4m3_words<T>(ld_shared_v4(raw + row * a.c.D + piece * 16),
                                          factor_of(e, T()), &lo, &hi);
                        st_shared_v4(dst + tile_chunk(row, piece * 2, X::kPanel), lo);
                        st_shared_v4(dst + tile_chunk(row, piece * 2 + 1, X::kPanel), hi);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        sv::mbar_arrive(&ctl.full[cs]);
                        sv::mbar_arrive(&ctl.raw_empty[rs]);
                    }
                }
            }
            ring += 2 * n;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // What join_kernel has to know: the item that this block began and did
        // not finish, and the block that did.
        Share sh{};
        sh.failed = *stop;
        sh.units = start.U;
        Walk<R> again(a, start);
        int64_t u = start.u0;
        while (again.next(&g)) {
            u += g.t.hi - g.t.lo;
            if (g.t.lo == g.item.lo && g.t.hi < g.item.hi) {
                const int64_t end = u + (g.item.hi - g.t.hi) - 1;  // the item's last unit
                int c = blockIdx.x + 1;
                while (share_begin(start.U, c + 1, gridDim.x) <= end) ++c;
                sh.leads = 1;
                sh.b = g.b;
                sh.h = g.h;
                sh.row0 = g.row0;
                sh.rows = g.rows;
                sh.q0 = g.q0;
                sh.last = c;
            }
        }
        args.shares[blockIdx.x] = sh;
    }
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

// Keys (kv = 0) or values (1) as [page][head][slot][element]; a box is the slots
// of one page in one tile, times 64 16-bit elements with the 128-byte swizzle or
// a whole row of codes.
bool make_map(CUtensorMap* map, const Cache& c, int kv, bool f16, bool e4m3)
{
    static const EncodeTiled fn = lookup_encode();
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

template <class T, int DP, bool E4M3, bool PAIR>
cudaError_t launch_shape(const CUtensorMap& k, const CUtensorMap& v, const Tiles& t, int blocks,
                         int64_t rows, cudaStream_t s)
{
    using X = Shape<DP, E4M3, PAIR>;
    constexpr size_t smem = X::kTiles + sizeof(Control<X::kStages, X::kRawStages, PAIR>);
    static_assert(smem <= kMaxSmem, "shared memory");
    auto* f = tiles_kernel<T, DP, E4M3, PAIR>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
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
    *mapped = make_map(&k, a.c, 0, f16, e4m3) && make_map(&v, a.c, 1, f16, e4m3);
    if (!*mapped) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    const int blocks = sms < kMaxBlocks ? sms : kMaxBlocks;
    const int64_t rows = item_rows(a.max_chunk, a.G);
    Tiles t{a, reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kShareBytes),
            static_cast<Share*>(workspace), static_cast<int32_t>(rows)};
    const bool pair = rows > 128;
    if (a.c.D <= 64)
        return f16 ? launch_type<F16, 64>(k, v, t, blocks, rows, e4m3, pair, s)
                   : launch_type<Bf16, 64>(k, v, t, blocks, rows, e4m3, pair, s);
    return f16 ? launch_type<F16, 128>(k, v, t, blocks, rows, e4m3, pair, s)
               : launch_type<Bf16, 128>(k, v, t, blocks, rows, e4m3, pair, s);
}

}  // namespace sva
