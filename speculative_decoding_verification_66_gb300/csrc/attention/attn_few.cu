// attn_few.cu -- attention over the paged cache by items of up to 16 rows: where a
// sequence has no more to a key/value head (a single token, a short draft), and for
// head sizes past 128, whose outputs would not fit attn_tiles.cu's tensor memory
// beside two slots' scores.
//
// Such items are bound by the reads of the cache: 2 D (1 + rows) operations meet
// 2 bytes of a key (or 1), far from the tensor cores' balance. The 128-row
// products of attn_tiles.cu would spend most of their time, and of the softmax
// warps' time, on rows that do not exist; here eight warps take 16 keys each of
// every 128-key tile, all rows, through m16n8k16 products in registers: the
// scores' accumulators are the weights' operands as they lie, no tile goes
// through tensor memory and no warp waits for another until the segment ends.
// A warp keeps a maximum, a sum and an output of its own for every row; they
// are joined through shared memory at the end of a segment.
//
// Measured: 512 single tokens, 500 to 2000 cached, 16 heads of 64: 467 us, 5.6 TB/s
// (with attn_tiles.cu 712 us); 4 tokens over 131000 e4m3 keys, 32 heads on 8: 233 us,
// 4.6 TB/s (300 us); the reads bound the first, the reads and the conversions the
// second (193 us with the loads alone). At 16 rows (64 x 4 tokens after 4000, 32 heads
// on 8) bfloat16 heads of 128 take 177 us here and 173 there, of 64 148 and 138, e4m3
// 173 and 190, 150 and 170. At 20 rows, which are two items here, 325 and 174, 268 and
// 140, e4m3 309 and 190, 275 and 170: up to 16, whatever the cache. Heads of 256: 64 x
// (1 to 5) tokens 344 us, a piece of 512 tokens after 3000 455 us (120 TFLOP/s).
//
// Warps 0-7 work, 8 and 9 load keys and values (attn_feed.cuh). Masks, hidden
// values and the sharing among blocks are those of attn_tiles.cu.
//
// e4m3. A lane reads 16 codes of a row at a time and expands them to float16 in
// registers. Keys: the codes alone (the exponents multiply the scores' columns);
// which d an operand's k slots stand for is free as long as the queries agree, so
// slots 2c, 2c+1, 2c+8, 2c+9 of step (h, s) are d = 16 (DP/64 c + h) + 4 s + 0..3,
// four neighbouring codes. Values, relative to their tile's largest exponent as in
// attn_tiles.cu: lane (g, c) reads d = DP/8 g .. of its four keys and interleaves
// the codes of two keys; the products' column n of step j is then d = DP/8 n + j.
#include "attn_feed.cuh"

namespace sva {
namespace {

constexpr int kWorkers = 8;
constexpr int kFewThreads = (kWorkers + 2) * 32;

template <int DP, bool E4M3>
struct FewShape {
    static constexpr int kRows = 16;
    static constexpr int kTileBytes = kTile * DP * (E4M3 ? 1 : 2);
    // Up to 192 KB of tiles.
    static constexpr int kMost = E4M3 ? 10 : 12;
    static constexpr int kStages = 196608 / kTileBytes < kMost ? 196608 / kTileBytes : kMost;
    static constexpr int kSteps = DP / 16;                  // products along d
    static constexpr int kQBytes = kSteps * 32 * 16;        // operands as the lanes hold them
    static constexpr int kJoin = 32;                        // columns joined at a time
    static constexpr int kJoinBytes = kWorkers * kRows * kJoin * 4;
    static constexpr int kBytes = kStages * kTileBytes + kQBytes + kJoinBytes;
};

template <int STAGES, bool E4M3>
struct FewControl {
    uint64_t full[STAGES], empty[STAGES], sync;
    uint64_t plan_ready[kItems];
    uint32_t filled[STAGES];  // how often the loads have filled a stage
    int stop;
    Start start;
    int64_t sums[kFewThreads / 32];
    Plan plan[kItems];
    int noted[kItems];
    int note[kItems][kNoted];
    int bad_page[kItems];
    uint32_t bad_rows[kWorkers];  // of a segment with pages out of range: by the warps
    float2 ml[kWorkers][16];
    float q_scale[16];
    // e4m3, for every stage: the keys' powers of two, or the values' factors as
    // halves and their largest exponent.
    alignas(16) float scale[E4M3 ? STAGES : 1][E4M3 ? kTile : 4];
    uint32_t top[E4M3 ? STAGES : 1];
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, Bf16)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, F16)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

template <class T, int DP, bool E4M3>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ Tiles args)
{
    using X = FewShape<DP, E4M3>;
    constexpr int S = X::kStages, R = X::kRows;
    using TP = typename std::conditional<E4M3, F16, T>::type;  // the products' operands
    const Attn& a = args.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    FewControl<S, E4M3>& ctl = *reinterpret_cast<FewControl<S, E4M3>*>(smem + X::kBytes);
    const uint32_t st = sv::smem_addr(smem), sq = st + S * X::kTileBytes;
    float* join = reinterpret_cast<float*>(smem + S * X::kTileBytes + X::kQBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    sv::pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            ctl.filled[i] = 0;
            sv::mbar_init(&ctl.full[i], 1);
            sv::mbar_init(&ctl.empty[i], kWorkers);
        }
        sv::mbar_init(&ctl.sync, kWorkers);
        for (int i = 0; i < kItems; ++i) sv::mbar_init(&ctl.plan_ready[i], 1);
        ctl.stop = (st & 1023u) != 0;  // (see attn_tiles.cu)
        for (int i = 0; i < kItems; ++i) ctl.noted[i] = ctl.bad_page[i] = 0;
        sv::fence_barrier_init();
    }
    if (find_start<R, kFewThreads>(a, ctl)) refuse_sequences<T, E4M3>(a, ctl);
    __syncthreads();
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
    if (warp >= kWorkers) {
        feed<T, DP, E4M3, R, false, false, S, true>(args, ctl, warp == kWorkers ? &kmap : &vmap,
                                              warp - kWorkers, st, X::kTileBytes, ctl.full, ctl.empty,
                                              start, wait_all);
    } else {
        const int g = lane >> 2, c4 = lane & 3;
        const float ninf = __uint_as_float(sv::kF32NegInfBits);
        uint32_t syncs = 0;
        // All eight warps come here; what they wrote before is seen after.
        auto meet = [&] {
            __syncwarp();
            if (lane == 0) sv::mbar_arrive(&ctl.sync);
            return wait_all(&ctl.sync, syncs++);
        };
        auto row_ptr = [&](const Plan& p, int r) {
            const int rr = p.row0 + r, t = rr / a.G;
            return a.q + (static_cast<int64_t>(p.q0) + t) * a.q_token +
                   static_cast<int64_t>(p.h * a.G + (rr - t * a.G)) * a.q_head;
        };
        // The queries' operands, as the lanes will hold them: step w by warp w.
        // Fetched into registers while a segment's results are joined, stored after.
        constexpr bool kScaled = E4M3 && std::is_same<T, Bf16>::value;
        constexpr int kPer = (X::kSteps + kWorkers - 1) / kWorkers;  // steps of a warp
        uint2 qv[kPer][2];    // rows g, g + 8
        uint2 qrow[kPer][2];  // kScaled: elements 4 lane .. (and from 128 on) of rows warp, warp + 8
        auto fetch = [&](const Plan& p) {
            if (kScaled) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = warp + 8 * i;
#pragma unroll
                    for (int z = 0; z < kPer; ++z) {
                        qrow[z][i] = make_uint2(0, 0);
                        if (r < p.rows && lane * 4 + 128 * z < a.c.D)
                            qrow[z][i] = *reinterpret_cast<const uint2*>(row_ptr(p, r) + lane * 8 +
                                                                         256 * z);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = g + 8 * i;
#pragma unroll
                for (int z = 0; z < kPer; ++z) {
                    const int step = warp + kWorkers * z;
                    qv[z][i] = make_uint2(0, 0);
                    if (step >= X::kSteps || r >= p.rows) continue;
                    const uint8_t* q = row_ptr(p, r);
                    if constexpr (E4M3) {
                        // step (h, s): d = 16 (DP/64 c + h) + 4 s
                        const int d = 16 * (DP / 64 * c4 + (step >> 2)) + 4 * (step & 3);
                        if (d < a.c.D) qv[z][i] = *reinterpret_cast<const uint2*>(q + d * 2);
                    } else if (16 * step < a.c.D) {
                        const int d = 16 * step + 2 * c4;
                        qv[z][i].x = *reinterpret_cast<const uint32_t*>(q + d * 2);
                        qv[z][i].y = *reinterpret_cast<const uint32_t*>(q + d * 2 + 16);
                    }
                }
            }
        };
        auto store = [&](int item) {
            if (kScaled) {
                // To float16: powers of two that bring a row's largest element to
                // [2^14, 2^15).
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t top = 0;
#pragma unroll
                    for (int z = 0; z < kPer; ++z) {
                        const uint2 u = qrow[z][i];
                        top = max(top, max(max(u.x << 16 & 0x7FFF0000u, u.x & 0x7FFF0000u),
                                           max(u.y << 16 & 0x7FFF0000u, u.y & 0x7FFF0000u)));
                    }
                    top = __reduce_max_sync(0xFFFFFFFFu, top);
                    if (lane == 0) {
                        const float size =
                            __uint_as_float(static_cast<uint32_t>(row_exponent(top) - 14) << 23);
                        ctl.q_scale[warp + 8 * i] = size;
                        row_factor(a.scale_log2 * size, &ctl.noted[item % kItems]);
                    }
                }
                if (!meet()) return false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t e = __float_as_uint(ctl.q_scale[g + 8 * i]) >> 23;
                    const float up = __uint_as_float((254u - e) << 23);
#pragma unroll
                    for (int z = 0; z < kPer; ++z) {
                        uint2& x = qv[z][i];
                        x.x = narrow2(sv::bf16_lo(x.x) * up, sv::bf16_hi(x.x) * up, F16());
                        x.y = narrow2(sv::bf16_lo(x.y) * up, sv::bf16_hi(x.y) * up, F16());
                    }
                }
            }
#pragma unroll
            for (int z = 0; z < kPer; ++z)
                if (warp + kWorkers * z < X::kSteps)
                    st_shared_v4(sq + ((warp + kWorkers * z) * 32 + lane) * 16,
                                 make_uint4(qv[z][0].x, qv[z][1].x, qv[z][0].y, qv[z][1].y));
            return meet();
        };
        Place<S> at;
        const Plan* plan = plan_at(ctl, 0, wait_all);
        if (plan != nullptr) fetch(*plan);
        bool ok = true;
        for (int item = 0; plan != nullptr; ++item) {
            const Plan& p = *plan;
            const int n = p.n, rows = p.rows;
            if (!(ok = store(item))) break;

            // This thread's rows: g + 8 i.
            int pos[2], low[2];
            float cs[2], m[2], l[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = min(g + 8 * i, rows - 1);
                pos[i] = p.cached + (p.row0 + r) / a.G;
                low[i] = p.low + (p.row0 + r) / a.G;
                cs[i] = a.scale_log2;
                if constexpr (E4M3 && std::is_same<T, Bf16>::value)
                    cs[i] = score_factor(cs[i] * ctl.q_scale[r]);
                m[i] = ninf;
                l[i] = 0.f;
            }
            float o[DP / 8][4];
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] = 0.f;

            int ref = 0;  // e4m3: the outputs' exponent
            for (int k = 0; k < n; ++k) {
                const bool edge = k < p.inner_lo || k > p.inner_hi;
                const int key0 = 16 * warp;  // this warp's keys of the tile
                // ---- scores: two products of eight keys side by side
                if (!(ok = wait_all(&ctl.full[at.stage], at.round))) break;
                const uint32_t kt = st + at.stage * X::kTileBytes;
                float s[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
                auto scores = [&](int step, const uint32_t (&b)[4]) {
                    const uint4 q = ld_shared_v4(sq + (step * 32 + lane) * 16);
                    const uint32_t f[4] = {q.x, q.y, q.z, q.w};
                    mma16816(s[0], f, b[0], b[1], TP());
                    mma16816(s[1], f, b[2], b[3], TP());
                };
                if constexpr (E4M3) {
#pragma unroll
                    for (int h = 0; h < DP / 64; ++h) {
                        uint4 w[2];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int row = key0 + 8 * t + g, ch = DP / 64 * c4 + h;
                            w[t] = make_uint4(0, 0, 0, 0);
                            if (ch * 16 < a.c.D)
                                w[t] = ld_shared_v4(kt + row * a.c.D +
                                                    few_swizzle<DP>(row, ch, args.swizzled) * 16);
                        }
                        const uint32_t w0[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
                        const uint32_t w1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint2 x = spread(w0[i]), y = spread(w1[i]);
                            const uint32_t b[4] = {x.x, x.y, y.x, y.y};
                            scores(4 * h + i, b);
                        }
                    }
                    // The keys' powers of two.
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 e = *reinterpret_cast<const float2*>(
                            &ctl.scale[at.stage][key0 + 8 * t + 2 * c4]);
                        s[t][0] *= e.x;
                        s[t][1] *= e.y;
                        s[t][2] *= e.x;
                        s[t][3] *= e.y;
                    }
                } else {
                    const int row = key0 + (lane & 7) + ((lane >> 4) << 3);
                    const uint32_t from = kt + row * 128;
                    const int y = ((lane >> 3) & 1) ^ (row & 7);
#pragma unroll
                    for (int step = 0; step < X::kSteps; ++step) {
                        uint32_t b[4];
                        ldmatrix4(from + (step >> 2) * kPanel + (((2 * (step & 3)) ^ y) << 4), b);
                        scores(step, b);
                    }
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.empty[at.stage]);
                at.advance(1);
                // ---- weights
                int lift = 0;  // e4m3: the tile's values above the outputs' exponent
                if (E4M3) {
                    // (the values' exponent comes with them)
                    if (!(ok = wait_all(&ctl.full[at.stage], at.round))) break;
                    const int v_top = static_cast<int>(ctl.top[at.stage]);
                    if (moves(ref, v_top)) {
                        const float keep = moved(ref, v_top);
#pragma unroll
                        for (int j = 0; j < DP / 8; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[j][i] *= keep;
                        ref = v_top;
                    }
                    lift = v_top > static_cast<int>(kLeast) ? v_top - ref : 0;
                }
                const float drop = E4M3 ? exp_value(static_cast<uint32_t>(127 - lift)) : 1.f;
                if (edge) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int x = k * kTile + key0 + 8 * t + 2 * c4 + i;
                            if (x < low[0] || x > pos[0]) s[t][i] = ninf;
                            if (x < low[1] || x > pos[1]) s[t][2 + i] = ninf;
                        }
                }
                bool grow = false;
                float top[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int z = 2 * i;
                    top[i] = fmaxf(fmaxf(s[0][z], s[0][z + 1]), fmaxf(s[1][z], s[1][z + 1])) * cs[i];
                    grow |= top[i] > m[i] + slack<T, E4M3>();
                }
                if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = top[i];
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
                        if (x > m[i] + slack<T, E4M3>()) {
                            x -= rise<T, E4M3>();
                            const float keep = sv::ex2(m[i] - x);
                            l[i] *= keep;
#pragma unroll
                            for (int j = 0; j < DP / 8; ++j) {
                                o[j][2 * i] *= keep;
                                o[j][2 * i + 1] *= keep;
                            }
                            m[i] = x;
                            if (too_far(x)) note_all(&ctl.noted[item % kItems]);
                        }
                    }
                }
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float shift = (m[i] == ninf ? 0.f : -m[i]) + static_cast<float>(lift);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float p0 = sv::ex2(fmaf(s[t][2 * i], cs[i], shift));
                        const float p1 = sv::ex2(fmaf(s[t][2 * i + 1], cs[i], shift));
                        l[i] = E4M3 ? fmaf(p0 + p1, drop, l[i]) : l[i] + (p0 + p1);
                        w[2 * t + i] = narrow2(p0, p1, TP());
                    }
                }
                // ---- values
                if (!E4M3 && !(ok = wait_all(&ctl.full[at.stage], at.round))) break;
                const uint32_t vt = st + at.stage * X::kTileBytes;
                if constexpr (E4M3) {
                    // Keys 2 c, 2 c + 1 and those eight further, as two pairs; up to
                    // 16 codes of a key at a time.
                    constexpr int kWords = DP == 64 ? 2 : 4;  // of four codes
                    const uint16_t* factor =
                        reinterpret_cast<const uint16_t*>(&ctl.scale[at.stage][0]) + key0 + 2 * c4;
                    const uint32_t f01 = *reinterpret_cast<const uint32_t*>(factor);
                    const uint32_t f23 = *reinterpret_cast<const uint32_t*>(factor + 8);
#pragma unroll
                    for (int part = 0; part < (DP == 256 ? 2 : 1); ++part) {
                        uint32_t codes[4][kWords];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int row = key0 + 2 * c4 + (z & 1) + 8 * (z >> 1);
                            const uint32_t from = vt + row * a.c.D;
                            if constexpr (DP >= 128) {
                                const int ch = DP / 128 * g + part;
                                uint4 x = make_uint4(0, 0, 0, 0);
                                if (ch * 16 < a.c.D)
                                    x = ld_shared_v4(from +
                                                     few_swizzle<DP>(row, ch, args.swizzled) * 16);
                                codes[z][0] = x.x, codes[z][1] = x.y;
                                codes[z][2] = x.z, codes[z][3] = x.w;
                            } else {
                                uint2 x = make_uint2(0, 0);
                                if (g * 8 < a.c.D)
                                    x = ld_shared_v2(from + (g & 1) * 8 +
                                                     few_swizzle<DP>(row, g >> 1, args.swizzled) * 16);
                                codes[z][0] = x.x, codes[z][1] = x.y;
                            }
                            // (a factor of zero: hidden, whatever the codes are)
                            if (edge && (((z >> 1 ? f23 : f01) >> (16 * (z & 1))) & 0xFFFFu) == 0u) {
#pragma unroll
                                for (int i = 0; i < kWords; ++i) codes[z][i] = 0;
                            }
                    }
#pragma unroll
                    for (int i = 0; i < kWords; ++i) {
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi) {
                            const int sel = hi ? 0x7362 : 0x5140;  // codes 2 hi, 2 hi + 1 of either key
                            const uint2 x = spread(__byte_perm(codes[0][i], codes[1][i], sel));
                            const uint2 y = spread(__byte_perm(codes[2][i], codes[3][i], sel));
                            const uint32_t x0 = mul2(x.x, f01), x1 = mul2(x.y, f01);
                            const uint32_t y0 = mul2(y.x, f23), y1 = mul2(y.y, f23);
                            mma16816(o[16 * part + 4 * i + 2 * hi], w, x0, y0, TP());
                            mma16816(o[16 * part + 4 * i + 2 * hi + 1], w, x1, y1, TP());
                        }
                    }
                    }
                } else {
                    if (edge) {
                        // Hidden values: see attn_tiles.cu.
                        constexpr int kLanes = DP / 8;  // lanes to a row
#pragma unroll 1
                        for (int x = lane; x < 16 * kLanes; x += 32) {
                            const int row = key0 + x / kLanes, ch = x % kLanes, q = k * kTile + row;
                            const uint32_t addr = vt + tile_chunk(row, ch);
                            const bool outside = q < p.any_lo || q > p.any_hi;
                            const bool common = q >= p.all_lo && q <= p.all_hi;
                            bool special = false;
                            if (!outside && !common)
                                special = any_special(ld_shared_v4(addr), exponent_mask(T()));
                            const unsigned mask = __ballot_sync(0xFFFFFFFFu, special) >>
                                                  (lane & ~(kLanes - 1));
                            const bool clear = (mask & ((1ull << kLanes) - 1)) != 0;
                            if (outside || clear) st_shared_v4(addr, make_uint4(0, 0, 0, 0));
                            if (clear && ch == 0) {
                                const int z = atomicAdd(&ctl.noted[item % kItems], 1);
                                if (z < kNoted) ctl.note[item % kItems][z] = q;
                            }
                        }
                        fence_async_smem();
                        __syncwarp();
                    }
                    const int row = key0 + (lane & 7) + (((lane >> 3) & 1) << 3);
                    const uint32_t from = vt + row * 128;
                    const int y = (lane >> 4) ^ (row & 7);
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j) {
                        uint32_t b[4];
                        ldmatrix4_trans(from + (j >> 2) * kPanel + (((2 * (j & 3)) ^ y) << 4), b);
                        mma16816(o[2 * j], w, b[0], b[1], TP());
                        mma16816(o[2 * j + 1], w, b[2], b[3], TP());
                    }
                }
                __syncwarp();
                if (lane == 0) sv::mbar_arrive(&ctl.empty[at.stage]);
                at.advance(1);
            }
            if (!ok) break;

            // ---- the warps' results joined
            plan = plan_at(ctl, item + 1, wait_all);
            if (plan != nullptr) fetch(*plan);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
                l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
                if (c4 == 0) ctl.ml[warp][g + 8 * i] = make_float2(m[i], l[i]);
            }
            const bool whole = p.whole != 0;
            const float nan = __uint_as_float(0x7FFFFFFFu);
            float* share = args.part + (static_cast<int64_t>(blockIdx.x) * 2 + (p.begins ? 1 : 0)) *
                                           args.part_rows * (DP + 4);
            // Every warp's rows, `width` columns of them from step j0 on, lie in
            // shared memory: added up, weighted, and written.
            int noted = 0;
            // Rows that see a position of a page out of range.
            uint32_t bad_rows = 0;
            if (*reinterpret_cast<volatile int*>(&ctl.bad_page[item % kItems]) != 0) {
                for (int r = warp; r < rows; r += kWorkers)
                    bad_rows |= meets_bad_page(a, p, r) ? 1u << r : 0u;
                if (lane == 0) ctl.bad_rows[warp] = bad_rows;
                if (!(ok = meet())) break;
                for (int i = 0; i < kWorkers; ++i) bad_rows |= ctl.bad_rows[i];
            }
            // A row that sees a noted position is computed again below.
            auto again = [&](int r) {
                if (noted == 0 || (bad_rows >> r & 1u)) return false;
                const int at_row = p.cached + (p.row0 + r) / a.G;
                const int from = p.low + (p.row0 + r) / a.G;
                bool x = noted > kNoted;
                for (int i = 0; i < min(noted, kNoted); ++i) {
                    const int q = *reinterpret_cast<volatile int*>(&ctl.note[item % kItems][i]);
                    x |= q >= from && q <= at_row;
                }
                return x;
            };
            auto add_up = [&](int j0, int width) {
                noted = *reinterpret_cast<volatile int*>(&ctl.noted[item % kItems]);
                const int steps = width >> 3;
                for (int x = threadIdx.x; x < rows * width; x += kWorkers * 32) {
                    const int r = x / width, y = x - r * width;
                    if (again(r)) continue;
                    const bool bad = (bad_rows >> r & 1u) != 0;
                    // e4m3: column n of step j is d = DP / 8 n + j
                    const int col = E4M3 ? y / steps : y & 7;
                    const int j = E4M3 ? y - col * steps : y >> 3;
                    const int d = E4M3 ? DP / 8 * col + j0 + j : 8 * j0 + y;
                    float top = ninf;
#pragma unroll
                    for (int w = 0; w < kWorkers; ++w) top = fmaxf(top, ctl.ml[w][r].x);
                    float sum = 0.f, total = 0.f;
#pragma unroll
                    for (int w = 0; w < kWorkers; ++w) {
                        const float2 z = ctl.ml[w][r];
                        const float weight = z.x == top ? 1.f : sv::ex2(z.x - top);
                        total = fmaf(z.y, weight, total);
                        sum = fmaf(join[(w * rows + r) * width + j * 8 + col], weight, sum);
                    }
                    const int rr = p.row0 + r, t = rr / a.G;
                    const int64_t orow = (static_cast<int64_t>(p.q0) + t) * a.Hq + p.h * a.G +
                                         (rr - t * a.G);
                    float* part = share + static_cast<int64_t>(r) * (DP + 4);
                    if (whole) {
                        if (d < a.c.D)
                            *reinterpret_cast<uint16_t*>(a.out + (orow * a.c.D + d) * 2) =
                                static_cast<uint16_t>(narrow2(bad ? nan : sum / total, 0.f, T()));
                        if (d == 0 && a.lse != nullptr)
                            a.lse[orow] = bad ? nan : fmaf(top, kLn2, logf(total));
                    } else {
                        part[d] = sum;
                        if (d == 0) {
                            part[DP] = top;
                            part[DP + 1] = bad ? nan : total;
                        }
                    }
                }
            };
            const float size = E4M3 && ref != 0 ? exp_value(static_cast<uint32_t>(ref)) * kDown : 1.f;
            // All columns at one time where they fit, else kJoin at a time.
            const bool once = rows * DP <= X::kRows * X::kJoin;
            const int width = once ? DP : X::kJoin;
            constexpr int kStepsJ = X::kJoin / 8;
#pragma unroll
            for (int j0 = 0; j0 < DP / 8; j0 += kStepsJ) {
                if (!once && j0 > 0 && !(ok = meet())) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (g + 8 * i >= rows) continue;
                    float* to = join + (warp * rows + g + 8 * i) * width + 2 * c4 + (once ? 8 * j0 : 0);
#pragma unroll
                    for (int j = 0; j < kStepsJ; ++j)
                        *reinterpret_cast<float2*>(to + j * 8) =
                            make_float2(o[j0 + j][2 * i] * size, o[j0 + j][2 * i + 1] * size);
                }
                if (!once) {
                    if (!(ok = meet())) break;
                    add_up(j0, width);
                }
            }
            if (ok && once && (ok = meet())) add_up(0, width);
            if (!ok) break;
            if (noted != 0) {
                for (int r = warp; r < rows; r += kWorkers) {
                    __syncwarp();
                    if (again(r))
                        again_row<T, E4M3, DP>(args, p, r, share + static_cast<int64_t>(r) * (DP + 4));
                }
            }
            __syncwarp();
            // (see attn_tiles.cu; every warp has read the notes of two segments ago)
            if (threadIdx.x == 0) {
                ctl.noted[(item + kItems - 2) % kItems] = 0;
                ctl.bad_page[(item + kItems - 2) % kItems] = 0;
            }
            // (what is read here is written again behind the next segment's store())
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) args.failed[blockIdx.x] = *stop;
    land<S>(ctl, ctl.full);
}

template <class T, int DP, bool E4M3>
cudaError_t launch_few_shape(const CUtensorMap& k, const CUtensorMap& v, const Tiles& t, int blocks,
                             int64_t rows, cudaStream_t s)
{
    using X = FewShape<DP, E4M3>;
    using Ctl = FewControl<X::kStages, E4M3>;
    constexpr size_t smem = X::kBytes + sizeof(Ctl);
    static_assert(smem <= kMaxSmem, "shared memory");
    static_assert(alignof(Ctl) == 16 && X::kBytes % 1024 == 0, "alignment");
    static_assert(X::kStages / 2 + 1 < kItems - 2, "notes");
    auto* f = few_kernel<T, DP, E4M3>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(f, smem, &allowed);
    if (e != cudaSuccess) return e;
    f<<<blocks, kFewThreads, smem, s>>>(k, v, t);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_join<T, DP>(t, blocks, rows, s);
}

template <class T, int DP>
cudaError_t launch_few_type(const CUtensorMap& k, const CUtensorMap& v, const Tiles& t, int blocks,
                            int64_t rows, bool e4m3, cudaStream_t s)
{
    return e4m3 ? launch_few_shape<T, DP, true>(k, v, t, blocks, rows, s)
                : launch_few_shape<T, DP, false>(k, v, t, blocks, rows, s);
}

}  // namespace

cudaError_t launch_attention_few(const Attn& a, bool f16, bool e4m3, void* workspace,
                                 cudaStream_t s)
{
    CUtensorMap k, v;
    Tiles t;
    int blocks = 0;
    const int64_t rows = a.max_chunk * a.G < kFewRows ? a.max_chunk * a.G : kFewRows;
    cudaError_t e = set_up(a, f16, e4m3, rows, workspace, true, &k, &v, &t, &blocks);
    if (e != cudaSuccess) return e;
    if (a.c.D <= 64)
        return f16 ? launch_few_type<F16, 64>(k, v, t, blocks, rows, e4m3, s)
                   : launch_few_type<Bf16, 64>(k, v, t, blocks, rows, e4m3, s);
    if (a.c.D <= 128)
        return f16 ? launch_few_type<F16, 128>(k, v, t, blocks, rows, e4m3, s)
                   : launch_few_type<Bf16, 128>(k, v, t, blocks, rows, e4m3, s);
    return f16 ? launch_few_type<F16, 256>(k, v, t, blocks, rows, e4m3, s)
               : launch_few_type<Bf16, 256>(k, v, t, blocks, rows, e4m3, s);
}

}  // namespace sva
