// lp_vec.cuh -- rows as 16-byte vectors, and packed arithmetic that CUDA C++ does
// not name.
#pragma once

#include "lp_common.cuh"

namespace svl {

template <int DT>
constexpr int kPerVec = DT == SV_F32 ? 4 : 8;      // elements of a vector
template <int DT>
constexpr int kElem = DT == SV_F32 ? 4 : 2;        // bytes of an element

// A row's 16-byte vectors, counted from the boundary at or below its first byte. Vector i
// holds elements i * kPerVec - head ..; those in [full, full_end) lie wholly in the row.
// The others (two at most) are moved element by element: nothing outside the row is
// touched.
struct Vecs {
    uint8_t* a0;
    int32_t head;      // elements between a0 and the row
    int32_t n;         // vectors
    int32_t full, full_end;
};

template <int DT>
__device__ __forceinline__ Vecs vectors_of(uint8_t* row, int32_t V)
{
    Vecs r;
    const uintptr_t p = reinterpret_cast<uintptr_t>(row);
    r.a0 = reinterpret_cast<uint8_t*>(p & ~uintptr_t(15));
    r.head = static_cast<int32_t>(p & 15) / kElem<DT>;
    const int64_t end = static_cast<int64_t>(r.head) + V;
    r.n = static_cast<int32_t>((end + kPerVec<DT> - 1) / kPerVec<DT>);
    r.full = r.head != 0;
    r.full_end = static_cast<int32_t>(end / kPerVec<DT>);
    return r;
}

// Index in the row of vector i's first element (negative for the first, with a head).
template <int DT>
__device__ __forceinline__ int64_t first_of(const Vecs& r, int32_t i)
{
    return static_cast<int64_t>(i) * kPerVec<DT> - r.head;
}

template <int DT>
constexpr uint32_t kNegInf = DT == SV_F32 ? 0xFF800000u : DT == SV_BF16 ? 0xFF80FF80u : 0xFC00FC00u;

// 16 bytes that are read once. (Not the read-only path: a gradient may be written over its
// logits.)
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// 16 bytes that are not read again here.
__device__ __forceinline__ void st_stream(uint8_t* p, uint4 v)
{
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// A vector that is not wholly in the row: -inf where it is not.
template <int DT>
__device__ __noinline__ uint4 ld_edge(const uint8_t* a0, int32_t i, int32_t head, int32_t V)
{
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        w[q] = kNegInf<DT>;
#pragma unroll
        for (int h = 0; h < kPerVec<DT> / 4; ++h) {
            const int64_t at = static_cast<int64_t>(i) * kPerVec<DT> + q * (kPerVec<DT> / 4) + h;
            if (at < head || at >= static_cast<int64_t>(head) + V) continue;
            if (DT == SV_F32) {
                w[q] = reinterpret_cast<const uint32_t*>(a0)[at];
            } else {
                const uint32_t b = reinterpret_cast<const uint16_t*>(a0)[at];
                w[q] = h == 0 ? (w[q] & 0xFFFF0000u) | b : (w[q] & 0x0000FFFFu) | (b << 16);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT>
__device__ __forceinline__ uint4 ld_vec(const Vecs& r, int32_t i, int32_t V)
{
    if (i >= r.full && i < r.full_end) return ld_stream(r.a0 + static_cast<int64_t>(i) * 16);
    if (i < r.n) return ld_edge<DT>(r.a0, i, r.head, V);
    return make_uint4(kNegInf<DT>, kNegInf<DT>, kNegInf<DT>, kNegInf<DT>);
}

// Pairs of floats in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t p, float& a, float& b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The elements of a vector as pairs of floats, exactly.
template <int DT>
__device__ __forceinline__ void widen(uint4 v, uint64_t (&p)[kPerVec<DT> / 2])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) {
        if (DT == SV_F32) {
            p[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else if (DT == SV_BF16) {
            p[i] = pack2(sv::bf16_lo(w[i]), sv::bf16_hi(w[i]));
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            p[i] = pack2(f.x, f.y);
        }
    }
}

// And back, each rounded once.
template <int DT>
__device__ __forceinline__ uint4 narrow(const uint64_t (&p)[kPerVec<DT> / 2])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < kPerVec<DT> / 2; ++i) {
        float a, b;
        unpack2(p[i], a, b);
        if (DT == SV_F32) {
            w[2 * i] = __float_as_uint(a);
            w[2 * i + 1] = __float_as_uint(b);
        } else if (DT == SV_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows that do not begin equally far from a boundary: vector j of the one (out) has its
// elements in vectors j + step and j + step + 1 of the other (in), `shift` elements on.
struct Shift {
    int32_t step, shift;
};
template <int DT>
__device__ __forceinline__ Shift shift_of(const Vecs& in, const Vecs& out)
{
    const int32_t d = in.head - out.head;
    return {d < 0 ? -1 : 0, d < 0 ? d + kPerVec<DT> : d};
}

// Bytes [by, by + 16) of the 32 in a and b.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, uint32_t by)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (by & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (by & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (by & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// A vector of results: whole, or the elements that lie in the row.
template <int DT>
__device__ __noinline__ void st_edge(uint8_t* a0, int32_t i, int32_t head, int32_t V, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < kPerVec<DT>; ++e) {
        const int64_t at = static_cast<int64_t>(i) * kPerVec<DT> + e;
        if (at < head || at >= static_cast<int64_t>(head) + V) continue;
        if (DT == SV_F32)
            reinterpret_cast<uint32_t*>(a0)[at] = w[e & 3];
        else
            reinterpret_cast<uint16_t*>(a0)[at] =
                static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
    }
}
template <int DT>
__device__ __forceinline__ void st_vec(const Vecs& r, int32_t i, int32_t V, uint4 v)
{
    if (i >= r.full && i < r.full_end)
        st_stream(r.a0 + static_cast<int64_t>(i) * 16, v);
    else if (i < r.n)
        st_edge<DT>(r.a0, i, r.head, V, v);
}

// Largest element of a vector (NaN if one is).
template <int DT>
__device__ __forceinline__ uint32_t packed_max(uint32_t a, uint32_t b)
{
    uint32_t r;
    if (DT == SV_F32)
        asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if (DT == SV_BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int DT>
__device__ __forceinline__ uint32_t vec_max(uint4 v)
{
    return packed_max<DT>(packed_max<DT>(v.x, v.y), packed_max<DT>(v.z, v.w));
}
template <int DT>
__device__ __forceinline__ float halves_max(uint32_t m)
{
    if (DT == SV_F32) return __uint_as_float(m);
    if (DT == SV_BF16) return fmax_nan(sv::bf16_lo(m), sv::bf16_hi(m));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return fmax_nan(f.x, f.y);
}

// Largest of a warp's floats (NaN if one is), to all lanes.
__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace svl
