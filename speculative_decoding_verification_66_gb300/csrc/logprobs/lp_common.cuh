// lp_common.cuh -- what the kernels over rows of logits share: descriptions of
// rows, element types, and small arithmetic.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "spec_verify.h"
#include "sv_device.cuh"
#include "sv_logprobs.h"

namespace svl {

using sv::ex2;
using sv::fmax_nan;

constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float inf() { return __uint_as_float(0x7F800000u); }
__device__ __forceinline__ float nan() { return __uint_as_float(0x7FFFFFFFu); }

// Where a row of an array [outer][inner][vocab] begins, in bytes.
struct RowAt {
    uint8_t* base;
    int64_t outer_bytes, inner_bytes;
};

struct Rows {
    RowAt x;
    int32_t inner;      // rows of one outer index
    int32_t rows;
    int32_t V;
    float c;            // log2(e) / T
    float inv_t;        // 1 / T
};

__device__ __forceinline__ uint8_t* row_begin(const RowAt& a, int32_t inner, int32_t row)
{
    const int32_t o = row / inner, i = row - o * inner;
    return a.base + o * a.outer_bytes + i * a.inner_bytes;
}

// One element, widened to float exactly; and a float rounded to the type once.
template <int DT>
__device__ __forceinline__ float load_one(const uint8_t* row, int64_t v)
{
    if (DT == SV_F32) return reinterpret_cast<const float*>(row)[v];
    const uint16_t h = reinterpret_cast<const uint16_t*>(row)[v];
    return DT == SV_BF16 ? __uint_as_float(static_cast<uint32_t>(h) << 16)
                         : __half2float(__ushort_as_half(h));
}

template <int DT>
__device__ __forceinline__ void store_one(uint8_t* row, int64_t v, float g)
{
    if (DT == SV_F32)
        reinterpret_cast<float*>(row)[v] = g;
    else if (DT == SV_BF16)
        reinterpret_cast<__nv_bfloat16*>(row)[v] = __float2bfloat16_rn(g);
    else
        reinterpret_cast<__half*>(row)[v] = __float2half_rn(g);
}

// Whole numbers in the floats' order (one zero; no NaN).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// log s for s > 0: the exponent's part is added in 64 bits, so that the error is that of a
// logarithm below 1/2 and not of one near 16.
__device__ __forceinline__ double log_wide(float s)
{
    if (!(s > 0.f && s < inf())) return static_cast<double>(logf(s));
    int e = 0;
    if (s < 1.1754944e-38f) {  // subnormal
        s *= 16777216.f;
        e = -24;
    }
    const uint32_t b = __float_as_uint(s);
    // s = 2^k f with f in [0.75, 1.5)
    const int k = (static_cast<int>(b) - 0x3F400000) >> 23;
    const float f = __uint_as_float(b - (static_cast<uint32_t>(k) << 23));
    return static_cast<double>(e + k) * 0.693147180559945309417 +
           static_cast<double>(log1pf(f - 1.0f));
}

}  // namespace svl
