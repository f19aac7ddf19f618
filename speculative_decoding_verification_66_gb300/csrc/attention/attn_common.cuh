// attn_common.cuh -- what the paged-cache and attention kernels share: the
// description of a cache and its chunks, element formats, and where a
// sequence's tokens lie.
#pragma once

#include <climits>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "sv_device.cuh"

namespace sva {

constexpr int kBadPage = 16;    // == SV_SEQ_BAD_PAGE
constexpr int kBadLength = 32;  // == SV_SEQ_BAD_LENGTH
constexpr int kTimeout = 4;     // == SV_SEQ_TIMEOUT
constexpr int kOverlap = 64;    // == SV_SEQ_OVERLAP

// Element types of the kernels' template parameters.
struct Bf16 {};
struct F16 {};

// A cache as the kernels see it: strides in bytes, the page size as a shift.
struct Cache {
    uint8_t* pages[2];
    uint8_t* exps[2];
    int64_t page_stride[2], slot_stride[2], head_stride[2];     // bytes
    int64_t exp_page_stride[2], exp_slot_stride[2], exp_head_stride[2];
    const int32_t* table;
    const int32_t* cached;
    const int32_t* starts;
    int64_t table_stride;
    int64_t capacity;  // max_pages * page_size: positions a table row can hold
    int32_t num_pages;
    int32_t page_shift;
    int32_t B, Hkv, D;
};

// A sequence's cached length and its rows of the packed arrays.
struct Seq {
    int64_t cached;
    int32_t start, count;
    int32_t bad;  // 0, kBadLength or kOverlap
};

__device__ __forceinline__ Seq seq_of(const Cache& c, int b, int64_t tokens, int64_t max_chunk)
{
    const int64_t s = c.starts[b], e = c.starts[b + 1];
    Seq q;
    q.cached = c.cached[b];
    const bool rows = s >= 0 && s <= e && e <= tokens;
    q.start = rows ? static_cast<int32_t>(s) : 0;
    q.count = rows ? static_cast<int32_t>(e - s) : 0;
    q.bad = (!rows || q.cached < 0 || e - s > max_chunk || q.cached + (e - s) > c.capacity)
                ? kBadLength
                : 0;
    return q;
}

// The sequence whose rows hold packed row t: the last b with starts[b] <= t,
// found by a warp 32 boundaries at a time (two steps up to 1024 sequences).
// The caller checks that row t is inside the sequence it gets, and, as the starts may
// be out of order, that it owns its rows.
//
// Sequence b owns its rows [s, e) if the search finds it for all of them, as it does
// where the starts are in order: if every step goes the same way for s and for e - 1,
// that is, if the boundaries taken (this lane's: *taken at most) are at most s and
// those behind them (*passed at least) at least e. So a row has one owner at most,
// whatever the starts are.
__device__ __forceinline__ int find_seq(const int32_t* starts, int B, int64_t t, int lane,
                                        int* taken, int* passed)
{
    int lo = 0, n = B;  // the answer is in [lo, lo + n)
    *taken = INT_MIN;
    *passed = INT_MAX;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool is = lane > 0 && lane * step < n;
        const int x = is ? starts[i] : INT_MIN;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, lane == 0 || (is && x <= t));
        const int k = 31 - __clz(static_cast<int>(m));  // lane 0 always votes
        if (lane == k) *taken = max(*taken, x);
        if (is && lane > k) *passed = min(*passed, x);
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

// Whether sequence b owns its rows [s, e), s < e, by a thread.
__device__ __forceinline__ bool owns_rows(const int32_t* starts, int B, int b, int64_t s, int64_t e)
{
    int lo = 0, n = B;
    while (n > 1) {
        const int step = (n + 31) / 32, k = (b - lo) / step;
        if (k > 0 && starts[lo + k * step] > s) return false;
        for (int j = k + 1; j < 32 && j * step < n; ++j)
            if (starts[lo + j * step] < e) return false;
        n = min(step, n - k * step);
        lo += k * step;
    }
    return true;
}
// seq_of, and kOverlap where some of the rows are not the sequence's own. A bad
// sequence's rows are those of its that lie in the packed arrays.
__device__ __forceinline__ Seq own_seq_of(const Cache& c, int b, int64_t tokens, int64_t max_chunk)
{
    Seq q = seq_of(c, b, tokens, max_chunk);
    if (!q.bad && q.count > 0 &&
        !owns_rows(c.starts, c.B, b, q.start, static_cast<int64_t>(q.start) + q.count))
        q.bad = kOverlap;
    if (q.bad) {
        const int64_t s = min(max(static_cast<int64_t>(c.starts[b]), int64_t(0)), tokens);
        const int64_t e = min(max(static_cast<int64_t>(c.starts[b + 1]), s), tokens);
        q.start = static_cast<int32_t>(s);
        q.count = static_cast<int32_t>(e - s);
    }
    return q;
}

// The page of position pos of sequence b, or -1 (outside [0, num_pages)).
__device__ __forceinline__ int32_t page_of(const Cache& c, int b, int64_t pos)
{
    const int32_t p = c.table[b * c.table_stride + (pos >> c.page_shift)];
    return p >= 0 && p < c.num_pages ? p : -1;
}

// Byte offset of (page, slot, head) in the keys (kv = 0) or values (kv = 1).
__device__ __forceinline__ int64_t vec_at(const Cache& c, int kv, int32_t page, int32_t slot, int h)
{
    return kv ? page * c.page_stride[1] + slot * c.slot_stride[1] + h * c.head_stride[1]
              : page * c.page_stride[0] + slot * c.slot_stride[0] + h * c.head_stride[0];
}
__device__ __forceinline__ int64_t exp_at(const Cache& c, int kv, int32_t page, int32_t slot, int h)
{
    return kv ? page * c.exp_page_stride[1] + slot * c.exp_slot_stride[1] + h * c.exp_head_stride[1]
              : page * c.exp_page_stride[0] + slot * c.exp_slot_stride[0] + h * c.exp_head_stride[0];
}

// 2^(e - 127) of an exponent byte in float32; NaN for 255. (0 means 2^-127, a
// subnormal; the library never writes less than 10.)
__device__ __forceinline__ float exp_value(uint32_t e)
{
    if (e == 255u) return __uint_as_float(0x7FFFFFFFu);
    return e == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

// Two packed 16-bit elements widened to float.
__device__ __forceinline__ float2 widen2(uint32_t w, Bf16)
{
    return make_float2(sv::bf16_lo(w), sv::bf16_hi(w));
}
__device__ __forceinline__ float2 widen2(uint32_t w, F16)
{
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(w));
    return f;
}

// Two floats rounded to nearest into packed 16-bit elements, a in the low half.
__device__ __forceinline__ uint32_t narrow2(float a, float b, Bf16)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, F16)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 codes (low byte first) to packed float16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
// Two floats to e4m3 codes, to nearest even, a in the low byte.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Eight consecutive cached elements as floats. E4M3: `p` points at the codes
// and `scale` is their power of two; otherwise 16-bit elements of type T.
template <class T, bool E4M3>
__device__ __forceinline__ void load8(const uint8_t* p, float scale, float (&f)[8])
{
    if (E4M3) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = ((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xFFFFu;
            const float2 v = widen2(e4m3_to_f16x2(two), F16());
            f[2 * i] = v.x * scale;
            f[2 * i + 1] = v.y * scale;
        }
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = widen2(u[i], T());
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

// Arguments of the attention kernels.
struct Attn {
    Cache c;
    const uint8_t* q;
    int64_t q_token, q_head;  // bytes
    uint8_t* out;             // [tokens, Hq, D]
    float* lse;               // [tokens, Hq] or nullptr
    int32_t* status;          // [B] or nullptr
    int64_t tokens, max_chunk, window;
    int32_t Hq, G;
    float scale;       // the caller's
    float scale_log2;  // scale * log2(e): softmax runs in powers of two
    // Test hook (nullptr in product calls): the values' loads of this thread block
    // (negative: of all) are held until *gate != 0.
    const int32_t* gate;
    int32_t gate_block;
};

constexpr float kLn2 = 0.693147180559945309f;

// First position that query position p sees.
__device__ __forceinline__ int64_t first_key(const Attn& a, int64_t p)
{
    return a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
}

// One query row against keys [lo, hi) of sequence b, by one warp, one key at a
// time: lane i holds elements 8 i .. 8 i + 7 of the query and of the output.
// On return m is the largest score in log2 units (-inf: none), l the sum of
// 2^(score - m) and o the weighted values, unnormalised. Returns false when a
// page is out of range.
template <class T, bool E4M3>
__device__ bool attend_row(const Attn& a, int b, int hkv, const uint8_t* q, int64_t lo, int64_t hi,
                           int lane, float* m_out, float* l_out, float (&o)[8])
{
    const Cache& c = a.c;
    const bool has = lane * 8 < c.D;
    const int eb = E4M3 ? 1 : 2;
    float x[8], m = __uint_as_float(sv::kF32NegInfBits), l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = o[i] = 0.f;
    if (has) load8<T, false>(q + lane * 16, 1.f, x);
    bool ok = true;
    for (int64_t j = lo; j < hi; ++j) {
        const int32_t page = page_of(c, b, j);
        if (page < 0) {
            ok = false;
            break;
        }
        const int32_t slot = static_cast<int32_t>(j) & ((1 << c.page_shift) - 1);
        float ks = 1.f, vs = 1.f;
        if (E4M3) {
            ks = exp_value(c.exps[0][exp_at(c, 0, page, slot, hkv)]);
            vs = exp_value(c.exps[1][exp_at(c, 1, page, slot, hkv)]);
        }
        float k[8], v[8], s = 0.f;
        if (has) {
            load8<T, E4M3>(c.pages[0] + vec_at(c, 0, page, slot, hkv) + lane * 8 * eb, ks, k);
            load8<T, E4M3>(c.pages[1] + vec_at(c, 1, page, slot, hkv) + lane * 8 * eb, vs, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(x[i], k[i], s);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s);  // a NaN score leaves m; its weight is NaN
        const float keep = m == mn ? 1.f : sv::ex2(m - mn);
        const float p = s == __uint_as_float(sv::kF32NegInfBits) ? 0.f : sv::ex2(s - mn);
        l = fmaf(l, keep, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = has ? fmaf(p, v[i], o[i] * keep) : 0.f;
        m = mn;
    }
    *m_out = m;
    *l_out = l;
    return ok;
}
// Its result as output row `row` of [tokens, Hq].
template <class T>
__device__ __forceinline__ void write_row(const Attn& a, int64_t row, int lane, float m, float l,
                                          const float (&o)[8])
{
    const float x = 1.f / l;
    if (lane * 8 < a.c.D)
        *reinterpret_cast<uint4*>(a.out + (row * a.c.D + lane * 8) * 2) =
            make_uint4(narrow2(o[0] * x, o[1] * x, T()), narrow2(o[2] * x, o[3] * x, T()),
                       narrow2(o[4] * x, o[5] * x, T()), narrow2(o[6] * x, o[7] * x, T()));
    if (a.lse != nullptr && lane == 0) a.lse[row] = fmaf(m, kLn2, logf(l));
}

}  // namespace sva
