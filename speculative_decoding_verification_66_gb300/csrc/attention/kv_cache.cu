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
// Both directions move bytes and little else. A vector (a token's key or value of
// one head) is moved by D / 8 lanes with 16-byte accesses of 8 elements, e4m3 by
// D / 16 lanes with 16 codes each. A warp takes one token, whose sequence and page
// it finds once for all its lanes, and kRounds rounds of as many vectors as fit
// side by side, with all its loads under way before the first is used. (More
// tokens a warp cost more in addresses of their own than they save: 58 us for
// 4 x 8000 tokens of 16 vectors against 43.)
#include "attn_internal.h"

namespace sva {
namespace {

constexpr int kThreads = 128;
constexpr int kRounds = 4;

// Largest magnitude with NaN and infinity kept: magnitudes order as their bits.
template <int N>
__device__ __forceinline__ uint32_t top_bits(const float (&f)[N])
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) t = max(t, __float_as_uint(f[i]) & 0x7FFFFFFFu);
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

template <class T>
__device__ __forceinline__ void unpack(uint4 w, float* f, T t)
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
__device__ __forceinline__ float limit(float f, Bf16) { return f; }
__device__ __forceinline__ float limit(float f, F16)
{
    return fabsf(f) < __uint_as_float(0x7F800000u) ? fminf(fmaxf(f, -61440.f), 61440.f) : f;
}

// LV lanes a vector (a power of two), `parts` warps a token.
template <class T, bool E4M3, bool READ, int LV>
__global__ void __launch_bounds__(kThreads) move_kernel(const Cache c, const Packed p, int parts)
{
    constexpr int kPer = E4M3 ? 16 : 8;  // elements a lane
    constexpr int kVecs = 32 / LV;       // vectors side by side
    const int lane = threadIdx.x & 31;
    // The blocks also report the sequences whose lengths are bad.
    if (p.status != nullptr)
        for (int64_t b = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; b < c.B;
             b += static_cast<int64_t>(gridDim.x) * kThreads) {
            const int bad = own_seq_of(c, static_cast<int>(b), p.tokens, p.tokens).bad;
            if (bad) atomicOr(p.status + b, bad);
        }
    const int64_t w = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = w / parts;
    const int part = static_cast<int>(w - t * parts);
    if (t >= p.tokens) return;
    int taken, passed;
    const int b = find_seq(c.starts, c.B, t, lane, &taken, &passed);
    const Seq q = seq_of(c, b, p.tokens, p.tokens);
    int32_t page = -1, slot = 0;
    if (!q.bad && t >= q.start && t - q.start < q.count &&
        __all_sync(0xFFFFFFFFu, taken <= q.start && passed - q.start >= q.count)) {
        const int64_t pos = q.cached + (t - q.start);
        page = page_of(c, b, pos);
        slot = static_cast<int32_t>(pos) & ((1 << c.page_shift) - 1);
        if (page < 0 && p.status != nullptr && lane == 0) atomicOr(p.status + b, kBadPage);
    }
    if (!READ && page < 0) return;
    const int n = 2 * c.Hkv;  // vectors of a token: keys' heads, then values'
    const int sub = lane & (LV - 1);
    const bool in_row = sub * kPer < c.D;
    // Where each round's vector lies.
    uint8_t* cache_at[kRounds];
    uint8_t* exp_at_[kRounds];
    uint8_t* row_at[kRounds];
    bool has[kRounds], ok[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
        const int v = (part * kRounds + u) * kVecs + lane / LV;
        const int kv = v >= c.Hkv ? 1 : 0, h = v - kv * c.Hkv;
        has[u] = v < n;
        ok[u] = has[u] && page >= 0;
        row_at[u] = (kv ? p.x[1] + t * p.token_stride[1] + h * p.head_stride[1]
                        : p.x[0] + t * p.token_stride[0] + h * p.head_stride[0]) + sub * kPer * 2;
        cache_at[u] = (kv ? c.pages[1] : c.pages[0]) + vec_at(c, kv, page, slot, h) + sub * 16;
        exp_at_[u] = E4M3 ? (kv ? c.exps[1] : c.exps[0]) + exp_at(c, kv, page, slot, h) : nullptr;
    }
    if constexpr (READ) {
        uint4 x[kRounds];
        uint32_t eb[kRounds];
        const uint32_t nan2 =
            narrow2(__uint_as_float(0x7FFFFFFFu), __uint_as_float(0x7FFFFFFFu), T());
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            x[u] = E4M3 ? make_uint4(0, 0, 0, 0) : make_uint4(nan2, nan2, nan2, nan2);
            eb[u] = 255;
            if (ok[u] && in_row) {
                x[u] = *reinterpret_cast<const uint4*>(cache_at[u]);
                if (E4M3) eb[u] = *exp_at_[u];
            }
        }
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            if (!has[u] || !in_row) continue;
            uint4* to = reinterpret_cast<uint4*>(row_at[u]);
            if (!E4M3) {
                to[0] = x[u];
                continue;
            }
            const float s = exp_value(eb[u]);
            const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = widen2(e4m3_to_f16x2((in[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), F16());
                o[i] = narrow2(f.x * s, f.y * s, T());
            }
            to[0] = make_uint4(o[0], o[1], o[2], o[3]);
            to[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    } else {
        uint4 x[kRounds][E4M3 ? 2 : 1];
#pragma unroll
        for (int u = 0; u < kRounds; ++u)
#pragma unroll
            for (int i = 0; i < (E4M3 ? 2 : 1); ++i)
                x[u][i] = ok[u] && in_row ? reinterpret_cast<const uint4*>(row_at[u])[i]
                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kRounds; ++u) {
            if constexpr (!E4M3) {
                if (ok[u] && in_row) *reinterpret_cast<uint4*>(cache_at[u]) = x[u][0];
            } else {
                float f[16];
                unpack(x[u][0], f, T());
                unpack(x[u][1], f + 8, T());
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = limit(f[i], T());
                uint32_t top = top_bits(f);
#pragma unroll
                for (int d = LV / 2; d > 0; d >>= 1)
                    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                if (!ok[u] || !in_row) continue;
                const uint32_t e = exp_byte(top);
                // 2^-(e - 127); a vector that is not finite keeps zero codes.
                const float inv = e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
                uint32_t q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = e == 255u ? 0u
                                     : f32_to_e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) |
                                           f32_to_e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16;
                *reinterpret_cast<uint4*>(cache_at[u]) = make_uint4(q[0], q[1], q[2], q[3]);
                if (sub == 0) *exp_at_[u] = static_cast<uint8_t>(e);
            }
        }
    }
}

template <class T, bool E4M3, bool READ, int LV>
cudaError_t launch_lanes(const Cache& c, const Packed& p, cudaStream_t s)
{
    constexpr int per = 32 / LV * kRounds;
    const int parts = (2 * c.Hkv + per - 1) / per;
    const int64_t work = (p.tokens * parts + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t blocks = work > 0 ? work : 1;  // (one for the statuses)
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    move_kernel<T, E4M3, READ, LV><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(c, p, parts);
    return cudaGetLastError();
}

template <class T, bool E4M3, bool READ>
cudaError_t launch_move(const Cache& c, const Packed& p, cudaStream_t s)
{
    // D is a multiple of 16 up to 256.
    const int lanes = c.D / (E4M3 ? 16 : 8);
    if (lanes <= 2) return launch_lanes<T, E4M3, READ, 2>(c, p, s);
    if (lanes <= 4) return launch_lanes<T, E4M3, READ, 4>(c, p, s);
    if (lanes <= 8) return launch_lanes<T, E4M3, READ, 8>(c, p, s);
    if (E4M3 || lanes <= 16) return launch_lanes<T, E4M3, READ, 16>(c, p, s);
    return launch_lanes<T, E4M3, READ, 32>(c, p, s);
}

template <bool READ>
cudaError_t launch_any(const Cache& c, const Packed& p, bool f16, bool e4m3, cudaStream_t s)
{
    if (c.B == 0) {
        // Rows of no sequence: NaN of either type.
        const size_t bytes = static_cast<size_t>(p.tokens) * c.Hkv * c.D * 2;
        cudaError_t e = cudaSuccess;
        for (int i = 0; READ && bytes > 0 && i < 2 && e == cudaSuccess; ++i)
            e = cudaMemsetAsync(p.x[i], 0xFF, bytes, s);
        return e;
    }
    if (p.tokens == 0 && p.status == nullptr) return cudaSuccess;
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
