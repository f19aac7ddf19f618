// kv_cache.cu -- writing new keys and values into the paged cache and reading
// ranges of it back.
//
// Writing to an SV_E4M3 cache: for a vector x with largest magnitude A,
//   e = max(ceil(log2(A / 448)), -117),  code_i = e4m3(x_i 2^-e).
// 448 = 1.75 2^8 is e4m3's largest value, so with A = f 2^k, 1 <= f < 2, e is
// k - 8 when f <= 1.75 and k - 7 otherwise: no logarithm and no division, and
// x 2^-e is exact, so the one rounding is the conversion (at most half a step,
// 2^-4 relative for values above 2^-6 2^e). A power of two costs nothing of a
// floating-point code's precision, and lets the attention kernels rebuild the
// stored value exactly in bfloat16.
//
// Both directions move bytes and little else. A warp takes one token and a
// group of its 2 Hkv vectors (keys' heads, then values'): each vector by
// D / 8 lanes with one 16-byte access of the 16-bit side, and kUnroll vectors
// a lane in flight before the first is used.
#include "attn_internal.h"

namespace sva {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;

// Largest magnitude with NaN and infinity kept: magnitudes order as their bits.
template <class T>
__device__ __forceinline__ uint32_t top_bits(const float (&f)[8])
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return t;
}

// The exponent byte of a vector whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t exp_byte(uint32_t top)
{
    if (top >= 0x7F800000u) return 255u;
    const int k = static_cast<int>(top >> 23) - 127;
    const int e = k - ((top & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return static_cast<uint32_t>(max(e, -117) + 127);
}

__device__ __forceinline__ void unpack(uint4 w, float (&f)[8], Bf16 t)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = widen2(u[i], t);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
__device__ __forceinline__ void unpack(uint4 w, float (&f)[8], F16 t)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = widen2(u[i], t);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
// float16 sources stay below 61440 = 240 2^8, so that no stored value rounds to
// 65536, which float16 does not have.
__device__ __forceinline__ void limit(float (&)[8], Bf16) {}
__device__ __forceinline__ void limit(float (&f)[8], F16)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (fabsf(f[i]) < __uint_as_float(0x7F800000u)) f[i] = fminf(fmaxf(f[i], -61440.f), 61440.f);
}

// Where warp `w` of the grid works.
struct Place {
    bool ok;       // the token's rows and page are good
    bool row;      // the token exists
    int64_t t;
    int32_t page, slot;
};

__device__ __forceinline__ Place place_of(const Cache& c, const Packed& p, int64_t t, int lane)
{
    Place w{false, t < p.tokens, t, -1, 0};
    if (!w.row) return w;
    const int b = find_seq(c.starts, c.B, t, lane);
    const Seq q = seq_of(c, b, p.tokens, p.tokens);
    if (q.bad || t < q.start || t - q.start >= q.count) return w;  // (status: status_kernel)
    const int64_t pos = q.cached + (t - q.start);
    w.page = page_of(c, b, pos);
    w.slot = static_cast<int32_t>(pos) & ((1 << c.page_shift) - 1);
    w.ok = w.page >= 0;
    if (!w.ok && p.status != nullptr && lane == 0) atomicOr(p.status + b, kBadPage);
    return w;
}

// LV lanes a vector (a power of two, 8 LV >= D).
template <class T, bool E4M3, bool READ, int LV>
__global__ void __launch_bounds__(kThreads) move_kernel(const Cache c, const Packed p, int parts)
{
    const int lane = threadIdx.x & 31;
    const int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    // The first blocks also report the sequences whose lengths are bad.
    if (p.status != nullptr)
        for (int64_t b = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; b < c.B;
             b += static_cast<int64_t>(gridDim.x) * kThreads) {
            const int bad = seq_of(c, static_cast<int>(b), p.tokens, p.tokens).bad;
            if (bad) atomicOr(p.status + b, bad);
        }
    const int64_t t = w / parts;
    const int part = static_cast<int>(w - t * parts);
    const Place at = place_of(c, p, t, lane);
    if (!at.row || (!READ && !at.ok)) return;
    constexpr int kVecs = 32 / LV;  // vectors a warp handles side by side
    const int sub = lane & (LV - 1);
    const bool has = sub * 8 < c.D;
    const int n = 2 * c.Hkv;
    const int v0 = part * kVecs * kUnroll + lane / LV;
    int64_t cache_off[kUnroll], exp_off[kUnroll], row_off[kUnroll];
    int kv[kUnroll];
    bool use[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int v = v0 + u * kVecs;
        use[u] = v < n;
        kv[u] = v >= c.Hkv ? 1 : 0;
        const int h = v - kv[u] * c.Hkv;
        cache_off[u] = vec_at(c, kv[u], at.page, at.slot, h) + sub * (E4M3 ? 8 : 16);
        exp_off[u] = E4M3 ? exp_at(c, kv[u], at.page, at.slot, h) : 0;
        row_off[u] = (kv[u] ? t * p.token_stride[1] + h * p.head_stride[1]
                            : t * p.token_stride[0] + h * p.head_stride[0]) + sub * 16;
    }
    if constexpr (READ) {
        uint4 r[kUnroll];
        uint2 codes[kUnroll];
        uint32_t eb[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t nan2 = narrow2(__uint_as_float(0x7FFFFFFFu), __uint_as_float(0x7FFFFFFFu), T());
            r[u] = make_uint4(nan2, nan2, nan2, nan2);
            codes[u] = make_uint2(0, 0);
            eb[u] = 255;
            if (use[u] && has && at.ok) {
                if (E4M3) {
                    codes[u] = *reinterpret_cast<const uint2*>((kv[u] ? c.pages[1] : c.pages[0]) + cache_off[u]);
                    eb[u] = (kv[u] ? c.exps[1] : c.exps[0])[exp_off[u]];
                } else {
                    r[u] = *reinterpret_cast<const uint4*>((kv[u] ? c.pages[1] : c.pages[0]) + cache_off[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!use[u] || !has) continue;
            if (E4M3) {
                const float s = exp_value(eb[u]);
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = ((i < 2 ? codes[u].x : codes[u].y) >> (16 * (i & 1))) & 0xFFFFu;
                    const float2 f = widen2(e4m3_to_f16x2(two), F16());
                    o[i] = narrow2(f.x * s, f.y * s, T());
                }
                r[u] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            *reinterpret_cast<uint4*>((kv[u] ? p.x[1] : p.x[0]) + row_off[u]) = r[u];
        }
    } else {
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        x[u] = use[u] && has ? *reinterpret_cast<const uint4*>((kv[u] ? p.x[1] : p.x[0]) + row_off[u])
                             : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (!E4M3) {
            if (use[u] && has) *reinterpret_cast<uint4*>((kv[u] ? c.pages[1] : c.pages[0]) + cache_off[u]) = x[u];
            continue;
        }
        float f[8];
        unpack(x[u], f, T());
        limit(f, T());
        uint32_t top = top_bits<T>(f);
#pragma unroll
        for (int d = LV / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if (!use[u] || !has) continue;
        const uint32_t e = exp_byte(top);
        // 2^-(e - 127); a vector that is not finite keeps zero codes.
        const float inv = e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = e == 255u ? 0u : f32_to_e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
        *reinterpret_cast<uint2*>((kv[u] ? c.pages[1] : c.pages[0]) + cache_off[u]) =
            make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        if (sub == 0) (kv[u] ? c.exps[1] : c.exps[0])[exp_off[u]] = static_cast<uint8_t>(e);
    }
    }
}

template <class T, bool E4M3, bool READ, int LV>
cudaError_t launch_lanes(const Cache& c, const Packed& p, cudaStream_t s)
{
    const int per = 32 / LV * kUnroll;
    const int parts = (2 * c.Hkv + per - 1) / per;
    const int64_t warps = p.tokens * parts;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    move_kernel<T, E4M3, READ, LV><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(c, p, parts);
    return cudaGetLastError();
}

template <class T, bool E4M3, bool READ>
cudaError_t launch_move(const Cache& c, const Packed& p, cudaStream_t s)
{
    // D is a multiple of 16 up to 256: 2 .. 32 lanes a vector.
    if (c.D <= 16) return launch_lanes<T, E4M3, READ, 2>(c, p, s);
    if (c.D <= 32) return launch_lanes<T, E4M3, READ, 4>(c, p, s);
    if (c.D <= 64) return launch_lanes<T, E4M3, READ, 8>(c, p, s);
    if (c.D <= 128) return launch_lanes<T, E4M3, READ, 16>(c, p, s);
    return launch_lanes<T, E4M3, READ, 32>(c, p, s);
}

template <bool READ>
cudaError_t launch_any(const Cache& c, const Packed& p, bool f16, bool e4m3, cudaStream_t s)
{
    if (p.tokens == 0 || c.B == 0) return cudaSuccess;
    if (!e4m3) return launch_move<Bf16, false, READ>(c, p, s);  // 16-bit elements move as they are
    return f16 ? launch_move<F16, true, READ>(c, p, s) : launch_move<Bf16, true, READ>(c, p, s);
}

}  // namespace

cudaError_t launch_append(const Cache& c, const Packed& p, bool f16, bool e4m3, cudaStream_t s)
{
    return launch_any<false>(c, p, f16, e4m3, s);
}
cudaError_t launch_read(const Cache& c, const Packed& p, bool f16, bool e4m3, cudaStream_t s)
{
    return launch_any<true>(c, p, f16, e4m3, s);
}

}  // namespace sva
