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
// last time: the weights stay below 2^slack(), which their type holds, and hardly any
// tile after the first needs it.
//
// P is rounded to the values' type, since a product's operands have to be of one type:
// by at most 2^-8 each in bfloat16, which takes the outputs' error from 0.0017 of their
// size, their own rounding, to 0.0023; in float16 (e4m3 caches too) by 2^-11, next to
// nothing. Two products, with P as the sum of two bfloat16, would take that away for
// half as much again of the tensor core's time.
//
// Two slots, each with its own S, O and softmax warpgroup, take turns on the
// tensor core: while one slot's rows go through the softmax, the other's
// products run.
//   PAIR    an item has up to 256 rows; slot s takes rows 128 s .. and both
//           use every tile of the item.
//   !PAIR   an item has up to 128 rows, both slots hold the same queries and
//           take every second tile; their results are joined at the end.
// PAIR halves the reads of a cache for chunks of more than 128 rows; !PAIR keeps
// the tensor core busy where there are fewer (launch_attention_tiles has the rule
// and what it rests on).
//
// Warps:
//   0-3, 4-7  softmax of slots 0 and 1 (row = tensor-memory lane = thread), the
//             loads of the queries and the outputs
//   8, 11     issue the products of slots 0 and 1. A warp's later instructions
//             queue behind the products it has issued, so one warp could not
//             look after one slot's barriers while the other's products run.
//   9, 10     load keys and values: page numbers, a bulk tensor copy a page,
//             exponents. Warp 9 also plans the block's segments for all.
//   12-..     helpers (4; e4m3: 8). 16-bit caches: make the values at a tile's
//             hidden positions harmless. e4m3 caches: expand every tile into the
//             stage that the products read.
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
// e4m3. Keys and values are expanded to float16, relative to the largest exponent
// of their tile (code_factor): 256 conversions and as many multiplications a tile
// and warp-width, where bfloat16 would take four times the instructions. The
// tile's exponents come back in where they cost nothing: the keys' in the scale of
// the tile's scores, the values' in the exponent of its weights, which are
// float16 too; O is kept relative to a reference exponent that follows the
// tiles'. Keys or values of a tile that are more than 2^22 apart would lose bits (a
// key that a row does not see could take them from those that it does); a segment
// that has such a tile computes its rows again, key by key. bfloat16
// queries become float16, each row scaled by a power of two that brings its
// largest element to [2^14, 2^15): exact down to 2^-38 of that.
//
// Work is shared among one block per SM as attn_plan.cuh says; items that
// several blocks share are joined by join_kernel in block order, so results
// depend on the lengths and the number of blocks alone.
//
// What bounds it. 16-bit drafts: the reads of the cache (64 x 5 tokens, contexts
// 1000 to 4000, 32 heads on 8: 123 us, 5.4 TB/s with both ends of a short call in
// it; 32 x (1 to 17), 8000 to 32768, 64 on 8: 436 us, 6.2 TB/s of 6.8). Pieces of
// prompts: the way from scores to weights to products, which the other slot covers
// in part (2048 tokens after 6000: 213 us, 1.11 PFLOP/s of 1.91; the tensor pipe
// runs half of the cycles). e4m3: the chain of loads, expansion, scores, weights and
// products, of which no part alone takes more than a sixth of the time (256 x 9:
// 660 us, 3.0 TB/s of codes, which are 6.0 TB/s of values; pieces of 1 to 700 tokens
// with a window: 169 us), and some 8 us from an item to the next.
#include "attn_feed.cuh"

namespace sva {
namespace {

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
    static constexpr int kRegsRow = 104, kRegsOther = 88, kRegsLaunch = 96;
    static_assert(8 * kRegsRow + 12 * kRegsOther <= 20 * kRegsLaunch, "registers");
    static constexpr int kTiles = kQBytes + kStages * kTileBytes + kRawStages * kRawBytes;
};

// Shared memory besides the tiles.
template <int STAGES, int RAW, bool PAIR>
struct Control {
    uint64_t full[STAGES], empty[STAGES], fixed[STAGES];
    uint64_t raw_full[RAW > 0 ? RAW : 1], raw_empty[RAW > 0 ? RAW : 1];
    uint64_t s_full[2], p_ready[2], q_ready, q_free, o_full, o_free, s_free, ml_ready, done;
    uint64_t plan_ready[kItems];
    uint32_t filled[RAW > 0 ? RAW : STAGES];  // how often the loads have filled a stage
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
    // .. of the last four tiles: the keys' power of two, the values' exponent
    float k_scale[4];
    int v_top[4];
    // e4m3, for every raw stage: the rows' factors; the exponents of its keys (or
    // values; plus 256: see kUnless) and of the values that belong to them.
    alignas(16) uint32_t factor[RAW > 0 ? RAW : 1][RAW > 0 ? kTile : 4];
    uint2 top[RAW > 0 ? RAW : 1];
};

template <class T, int DP, bool E4M3, bool PAIR>
__global__ void __launch_bounds__(Shape<DP, E4M3, PAIR>::kThreads, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ Tiles args)
{
    using X = Shape<DP, E4M3, PAIR>;
    constexpr int S = X::kStages, RS = X::kRawStages, R = X::kRows;
    constexpr int kFill = E4M3 ? RS : S;  // stages that the copies fill
    using TP = typename std::conditional<E4M3, F16, T>::type;  // the products' operands
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
        for (int i = 0; i < kFill; ++i) ctl.filled[i] = 0;
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

    if (find_start<R, X::kThreads>(a, ctl)) refuse_sequences<T, E4M3>(a, ctl);
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

    if (E4M3 && warp >= 8)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kRegsOther));
    if (warp < 8) {
        // ------------------------------------------------------------------
        // Softmax of slot s; thread = row.
        // ------------------------------------------------------------------
        if (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(X::kRegsRow));
        const int s = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        // Columns of scores in registers at a time: 64 wait for fewer loads (when
        // this was chosen, a 2048-token piece 222 us against 228 with 32); e4m3 has
        // more code to keep in the instruction caches and fewer registers (256 x 9:
        // 668 us with 32, 724 with 64 and 120 registers, which spill).
        constexpr bool kWide = !E4M3;
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
        // From a row to the one that is kStep further, in tokens and heads.
        constexpr int kStep = 128 / kChunks;
        const int step_t = kStep / a.G, step_h = kStep - step_t * a.G;
        auto fetch = [&](const Plan& x) {
            int t = (x.row0 + first) / a.G, head = x.row0 + first - t * a.G;
#pragma unroll
            for (int i = 0; i < kFetch; ++i) {
                qv[i] = make_uint4(0, 0, 0, 0);
                if (first + i * kStep < x.rows && ch * 8 < a.c.D)
                    qv[i] = *reinterpret_cast<const uint4*>(
                        a.q + (static_cast<int64_t>(x.q0) + t) * a.q_token +
                        static_cast<int64_t>(x.h * a.G + head) * a.q_head + ch * 16);
                t += step_t;
                head += step_h;
                if (head >= a.G) {
                    head -= a.G;
                    ++t;
                }
            }
        };
        auto store = [&](const Plan& x, int at) {
#pragma unroll
            for (int i = 0; i < kFetch; ++i) {
                const int r = first + i * kStep;
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
                    const int e = row_exponent(top);
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
                                     tile_chunk(r & 127, ch),
                                 qv[i]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) sv::mbar_arrive(&ctl.q_ready);
        };

        const Plan* ahead = plan_at(ctl, 0, wait_all);
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
            int ref = 0;  // e4m3: O's exponent
            bool begun = false;
            {
                // The last position that the row sees, and the first.
                const int of = (g.row0 + min(slot_row, rows - 1)) / a.G;
                const int pos = g.cached + of, low = g.low + of;
                const int k0 = PAIR ? (s ? g.lo1 : g.lo0) : s;
                const int k1 = PAIR ? (s ? g.hi1 : g.hi0) : g.n;
                float row_c = a.scale_log2, c = row_c;
                for (int k = k0; k < k1; k += PAIR ? 1 : 2) {
                    if (!(ok = wait_all(&ctl.s_full[s], tiles_done))) break;
                    ++tiles_done;
                    if (live) {
                        fence_after();
                        if (E4M3 && std::is_same<T, Bf16>::value && !begun)
                            row_c = row_factor(
                                a.scale_log2 * ctl.q_scale[item & 1][min(slot_row, rows - 1)],
                                &ctl.noted[item % kItems]);
                        const int clo = low - k * kTile, chi = pos - k * kTile;
                        const bool masked =
                            __any_sync(0xFFFFFFFFu, clo > 0 || chi < kTile - 1) != 0;
                        // The loops below are kept rolled: all roles' code has to
                        // stay in the instruction caches.
                        int lift = 0;  // e4m3: the tile's values above O's exponent
                        bool move = false;
                        float keep_v = 1.f;
                        if (E4M3) {
                            c = score_factor(row_c * ctl.k_scale[(tiles_before + k) & 3]);
                            const int top = ctl.v_top[(tiles_before + k) & 3];
                            if ((move = moves(ref, top))) {
                                keep_v = moved(ref, top);
                                ref = top;
                            }
                            lift = top > static_cast<int>(kLeast) ? top - ref : 0;
                        }
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
                        // 32 or (kWide) 64 columns at a time.
                        float v[32], v2[32], mt = ninf;
#pragma unroll 1
                        for (int x = 0; x < kTile; x += kWide ? 64 : 32)
                            mt = fmaxf(mt, kWide ? tmem_ld_max(s_addr + x, v, s_addr + x + 32, v2)
                                                 : tmem_ld_max(s_addr + x, v));
                        // (scale > 0; a NaN score is left out here and comes through below)
                        mt *= c;
                        const bool grow = mt > m + slack<T, E4M3>() || (!begun && mt > m);
                        if (begun && __any_sync(0xFFFFFFFFu, grow || move)) {
                            // The slot's products so far are complete: s_full's
                            // commit came after them.
                            const float keep = grow ? sv::ex2(m - (mt - rise<T, E4M3>())) : 1.f;
#pragma unroll 1
                            for (int x = 0; x < DP / 16; ++x) {
                                float o[16];
                                tmem_ld(o_addr + 16 * x, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= keep * keep_v;
                                tmem_st(o_addr + 16 * x, o);
                            }
                            l *= keep;
                        }
                        if (grow) {
                            m = mt - rise<T, E4M3>();
                            // (lanes without a row have scores of whatever lies in its place)
                            if (too_far(m) && slot_row < rows) note_all(&ctl.noted[item % kItems]);
                        }
                        begun = true;
                        const float shift = (m == ninf ? 0.f : -m) + static_cast<float>(lift);
                        float2 l0 = make_float2(0.f, 0.f), l1 = l0;
                        auto weigh = [&](const float (&y)[32], int x) {
                            uint32_t w[16];
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float2 p = fma2(make_float2(y[2 * i], y[2 * i + 1]), c, shift);
                                float2 q = fma2(make_float2(y[2 * i + 2], y[2 * i + 3]), c, shift);
                                p = make_float2(sv::ex2(p.x), sv::ex2(p.y));
                                q = make_float2(sv::ex2(q.x), sv::ex2(q.y));
                                l0 = add2(l0, p);
                                l1 = add2(l1, q);
                                w[i] = narrow2(p.x, p.y, TP());
                                w[i + 1] = narrow2(q.x, q.y, TP());
                            }
                            tmem_st(s_addr + 64 + x / 2, w);
                        };
                        // The weights, the last columns first: they take the columns
                        // of the upper half from the top.
#pragma unroll 1
                        for (int x = kTile - (kWide ? 64 : 32);;) {
                            weigh(v, x);
                            if (kWide) weigh(v2, x + 32);
                            if (x == 0) break;
                            x -= kWide ? 64 : 32;
                            if (kWide)
                                tmem_ld(s_addr + x, v, s_addr + x + 32, v2);
                            else
                                tmem_ld(s_addr + x, v);
                        }
                        const float sum = (l0.x + l0.y) + (l1.x + l1.y);
                        l += E4M3 ? sum * exp_value(static_cast<uint32_t>(127 - lift)) : sum;
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
            ahead = plan_at(ctl, item + 1, wait_all);
            if (ahead != nullptr) {
                fetch(*ahead);
                if (!(ok = wait_all(&ctl.q_free, item))) break;
                store(*ahead, item + 1);
            }
            if (!(ok = wait_all(&ctl.o_full, item))) break;
            fence_after();
            // O's true size: e4m3, its reference exponent.
            const float size = E4M3 && ref != 0 ? exp_value(static_cast<uint32_t>(ref)) * kDown : 1.f;
            float w0 = size, w1 = 0.f;
            if (!PAIR) {
                // The slots exchange their rows' maxima and sums through the
                // scores' columns, which the products have done with.
                if (live) {
                    tmem_st4(s_addr, m, l, size, 0.f);
                    tmem_wait_st();
                    fence_before();
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.ml_ready);
                if (!(ok = wait_all(&ctl.ml_ready, item))) break;
                if (live) {
                    fence_after();
                    float om, ol, osize, none;
                    tmem_ld4(lane_base + (1 - s) * 128, om, ol, osize, none);
                    fence_before();
                    const float top = fmaxf(m, om);
                    const float wm = m == top ? 1.f : sv::ex2(m - top);
                    const float wo = om == top ? 1.f : sv::ex2(om - top);
                    // (the same order in both slots)
                    l = (s ? ol * wo : l * wm) + (s ? l * wm : ol * wo);
                    w0 = s ? wo * osize : wm * size;
                    w1 = s ? wm * size : wo * osize;
                    m = top;
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.s_free);
            }
            const bool whole = g.whole != 0, valid = slot_row < rows;
            // A row that sees a noted position is computed again below.
            const int noted = *reinterpret_cast<volatile int*>(&ctl.noted[item % kItems]);
            const bool bad = *reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) != 0 &&
                             meets_bad_page(a, g, min(slot_row, rows - 1));
            const int r = g.row0 + min(slot_row, rows - 1), token = r / a.G;
            bool again = noted > kNoted;
            if (noted > 0) {
                const int pos = g.cached + token, low = g.low + token;
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
                // Columns of the row, 32 at a time (more of both slots' would not
                // stay in registers): all, or the slot's half where both slots hold
                // the row.
                constexpr int kCols = 32;
                const int64_t orow = (static_cast<int64_t>(g.q0) + token) * a.Hq + g.h * a.G +
                                     (r - token * a.G);
                const float inv = bad ? nan : (whole ? 1.f / l : 1.f) * (PAIR ? size : 1.f);
                float* part = share + static_cast<int64_t>(slot_row) * (DP + 4);
#pragma unroll 1
                for (int x = 0; x < DP / (PAIR ? kCols : 2 * kCols); ++x) {
                    const int k0 = (PAIR ? 0 : s * (DP / 2)) + kCols * x;
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
                        for (int i = 0; i < kCols; ++i) o[i] = n > 1 ? o[i] * w0 + p[i] * w1 : o[i] * w0;
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
    } else if (warp == 8 || warp == 11) {
        // ------------------------------------------------------------------
        // Products of slot s: the warp stays together, one lane issues. It
        // passes every tile in ring order, its own and the other slot's.
        // ------------------------------------------------------------------
        constexpr uint32_t id_s = idesc<TP, kTile, false>(), id_o = idesc<TP, DP, true>();
        const int s = warp == 8 ? 0 : 1;
        const uint64_t dq = smem_desc(sq + (PAIR ? s * (128 * DP * 2) : 0), 16, 1024);
        const uint64_t dk = smem_desc(st, 16, 1024), dv = smem_desc(st, kPanel, 1024);
        constexpr uint32_t panel = kPanel >> 4, v_step = 2048 >> 4;  // 16 keys: two groups of 8
        const uint32_t s_addr = tmem + s * 128, o_addr = tmem + 256 + s * DP;
        Place<S> at;
        uint32_t fixes = 0, tiles = 0;
        bool ok = true;
        for (; ok; ++item) {
            const Plan* g = plan_at(ctl, item, wait_all);
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
                const bool is_v = vv < n && ring_v<!PAIR>(vv, n) == i;
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
                    auto keys_here = [&] {
                        return __all_sync(0xFFFFFFFFu,
                                          mbar_test(&ctl.full[keys.stage], keys.round & 1u)) != 0;
                    };
                    if (left > 0) scores = keys_here();
                    if (!(ok = wait_all(&ctl.p_ready[s], tiles))) break;
                    if (left > 0 && !scores) scores = keys_here();
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
                                mma_ss(s_addr, dq + o + (x >> 2) * panel,
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
        // Copies of keys (warp 9, which also plans the segments) and values (10).
        feed<T, DP, E4M3, R, PAIR, !PAIR, kFill, false>(
            args, ctl, warp == 9 ? &kmap : &vmap, warp - 9, E4M3 ? sr : st,
            E4M3 ? X::kRawBytes : X::kTileBytes, E4M3 ? ctl.raw_full : ctl.full,
            E4M3 ? ctl.raw_empty : ctl.empty, start, wait_all);
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
            const Plan* g = plan_at(ctl, item, wait_all);
            if (g == nullptr) break;
            const int n = g->n, inner_lo = g->inner_lo, inner_hi = g->inner_hi;
            auto note = [&](int p) {
                const int i = atomicAdd(&ctl.noted[item % kItems], 1);
                if (i < kNoted) ctl.note[item % kItems][i] = p;
            };
            int kk = 0, vv = 0;
            for (int i = 0; ok && i < 2 * n; ++i) {
                const bool is_v = vv < n && ring_v<!PAIR>(vv, n) == i;
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
                            const uint32_t addr = v + tile_chunk(row, ch);
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
                    // kStep-th row, four at a time. Eight neighbouring lanes take half
                    // of the pieces of two rows, the other half of the second: their
                    // 16-byte columns differ in the loads and, swizzled, in the stores.
                    constexpr int kPieces = DP / 16, kStep = kThreadsH / kPieces;
                    const int pair = tid / (2 * kPieces), odd = (tid >> 2) & 1;
                    const int row0 = pair * 2 + odd;
                    const int piece = (tid & 3) + (kPieces > 4 ? (((tid >> 3) & 1) ^ odd) << 2 : 0);
                    const bool in_row = piece * 16 < a.c.D;
                    const uint32_t from = raw + row0 * a.c.D + (in_row ? piece * 16 : 0);
                    const uint32_t to = dst + tile_chunk(row0, piece * 2);
                    const uint32_t* factor = &ctl.factor[raw_at.stage][row0];
                    if (!is_v && tid == 0) {
                        const uint2 top = ctl.top[raw_at.stage];
                        ctl.k_scale[k_tiles & 3] = exp_value(top.x & 255u) * kDown;
                        ctl.v_top[k_tiles & 3] = static_cast<int>(top.y);
                    }
                    const bool ragged = k < inner_lo || k > inner_hi;
                    constexpr int kBatch = kTile / kStep < 4 ? kTile / kStep : 4;
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
                            // (a factor of zero: hidden, whatever the codes are)
                            if (ragged && f[u] == 0u) codes[u] = make_uint4(0, 0, 0, 0);
                            uint32_t o[8];
                            expand(codes[u], f[u], o);
                            // (chunk 2 c + 1 is chunk 2 c's neighbour under the swizzle too)
                            const uint32_t t = to + (r + u * kStep) * 128;
                            st_shared_v4(t, make_uint4(o[0], o[1], o[2], o[3]));
                            st_shared_v4(t ^ 16u, make_uint4(o[4], o[5], o[6], o[7]));
                        }
                    }
                    if (ctl.top[raw_at.stage].x >= 256u && in_row) {
                        // (every thread those that it has expanded)
#pragma unroll 1
                        for (int row = 0; row < kTile; row += kStep)
                            if (factor[row] == both(kUnless) &&
                                not_zeros(ld_shared_v4(from + row * a.c.D)))
                                atomicAdd(&ctl.noted[item % kItems], kNoted + 1);
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
    __syncthreads();
    if (threadIdx.x == 0) args.failed[blockIdx.x] = *stop;
    land<kFill>(ctl, E4M3 ? ctl.raw_full : ctl.full);
    if (warp == 8) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
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
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(f, smem, &allowed);
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
    return launch_join<T, DP>(t, blocks, rows, s);
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
int64_t item_rows(int64_t max_chunk, int64_t G, int64_t most)
{
    return max_chunk * G < most ? max_chunk * G : most;
}

}  // namespace

size_t tiles_workspace(int64_t max_chunk, int64_t G, int64_t D)
{
    const int64_t dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    const int64_t rows = item_rows(max_chunk, G, D <= kMaxTileDim ? 256 : kFewRows);
    return kShareBytes + kFailedBytes +
           static_cast<size_t>(kMaxBlocks) * 2 * rows * (dp + 4) * sizeof(float);
}

cudaError_t launch_attention_tiles(const Attn& a, bool f16, bool e4m3, void* workspace,
                                   cudaStream_t s)
{
    CUtensorMap k, v;
    Tiles t;
    int blocks = 0;
    // PAIR where the sequences have more than 128 rows on average (their number is
    // known, their lengths are not). 64 x 33 tokens of 4 heads after 4000: 262 us
    // with, 338 without, 64 x 64: 269 and 353, a piece of 2048: 214 and 228; chunks
    // from 1 to 33: 165 and 138, 32 x (1 to 17) of 8 heads: 476 and 440: items of up
    // to 128 rows leave the second slot idle.
    const bool pair = a.max_chunk * a.G > 128 && a.tokens * a.G > 128 * static_cast<int64_t>(a.c.B);
    const int64_t rows = item_rows(a.max_chunk, a.G, pair ? 256 : 128);
    cudaError_t e = set_up(a, f16, e4m3, rows, workspace, false, &k, &v, &t, &blocks);
    if (e != cudaSuccess) return e;
    if (a.c.D <= 64)
        return f16 ? launch_type<F16, 64>(k, v, t, blocks, rows, e4m3, pair, s)
                   : launch_type<Bf16, 64>(k, v, t, blocks, rows, e4m3, pair, s);
    return f16 ? launch_type<F16, 128>(k, v, t, blocks, rows, e4m3, pair, s)
               : launch_type<Bf16, 128>(k, v, t, blocks, rows, e4m3, pair, s);
}

}  // namespace sva
