// The 4-bit row format (KVC_Q4, see kvc.h), shared by every kernel that reads
// or writes it.
//
// A row is one token of one KV head, K and V apart: d codes of 4 bits, eight
// to a 32-bit word (value 2i at bits 4i, value 2i + 1 at bits 16 + 4i), and
// one scale word (bf16 step s in the high 16 bits, zero point z in the low
// 16).  A value is s * (c - z).
//
// Why this order in a word: w & 0x000F000F, (w >> 4) & 0x000F000F, ... are then
// pairs of neighbouring values, one per 16-bit half, which is how the packed
// 16-bit arithmetic and the matrix fragments want them.  Why one step a row: a
// row's step multiplies a whole dot product (K) or a whole softmax weight (V),
// so attention never rescales single values.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "kvc_internal.h"

namespace kvc {
namespace q4 {

constexpr float kMinStep = 1.17549435e-38f;  // 2^-126: a smaller step stores the row as zeros

__device__ __forceinline__ float step_of(uint32_t scale_word) { return __uint_as_float(scale_word & 0xFFFF0000u); }
__device__ __forceinline__ int zero_of(uint32_t scale_word) { return static_cast<int>(scale_word & 0xFFFFu); }

// Code of value e (0 .. 7) of a word.
__device__ __forceinline__ int code_of(uint32_t w, int e) { return (w >> (((e & 1) << 4) + ((e >> 1) << 2))) & 15; }

// lo = min(0, x), hi = max(0, x) over eight bf16 values; a NaN or an infinity
// among them gives hi = +inf, so that the row's range is not finite.
__device__ __forceinline__ void range8(const uint32_t (&w)[4], float& lo, float& hi) {
    lo = hi = 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
        lo = fminf(lo, fminf(a, b));
        hi = fmaxf(hi, fmaxf(a, b));
        top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    }
    if (top >= 0x7F80u) hi = INFINITY;
}

// A row's step, reciprocal and zero point from its range, in the format's
// float32 operations; the row is stored as zeros (step 0) or as NaN (step NaN)
// when `plain` comes back false.
struct RowScale {
    float inv;
    int z;
    uint32_t word;
    bool plain;
};
__device__ __forceinline__ RowScale row_scale(float lo, float hi) {
    RowScale r;
    const float span = __fsub_rn(hi, lo);
    const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(span, 15.f)));
    const bool finite = span <= 3.402823466e38f;
    r.plain = finite && s >= kMinStep;
    r.inv = r.plain ? __frcp_rn(s) : 0.f;
    r.z = r.plain ? __float2int_rn(__fmul_rn(-lo, r.inv)) : 0;
    r.word = r.plain ? (__float_as_uint(s) | static_cast<uint32_t>(r.z)) : (finite ? 0u : 0x7FC00000u);
    return r;
}

// The code word of eight bf16 values of a row.
__device__ __forceinline__ uint32_t encode8(const uint32_t (&w)[4], const RowScale& r) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = __float2int_rn(__fmul_rn(__uint_as_float(w[i] << 16), r.inv)) + r.z;
        const int b = __float2int_rn(__fmul_rn(__uint_as_float(w[i] & 0xFFFF0000u), r.inv)) + r.z;
        out |= static_cast<uint32_t>(min(15, max(0, a))) << (4 * i);
        out |= static_cast<uint32_t>(min(15, max(0, b))) << (16 + 4 * i);
    }
    return r.plain ? out : 0u;
}

// Index of a cache row's scale word: rows are numbered unit * tokens + offset
// (a unit is one KV head of a batch row or of a page) and a unit's scale words
// take `stride` = tokens rounded up to a multiple of 4, so that every unit's
// words start on a 16-byte boundary.
__device__ __forceinline__ size_t scale_index(const Q4Scales& sc, int row) {
    if (sc.stride == sc.tokens) return static_cast<size_t>(row);
    const int unit = row / sc.tokens;
    return static_cast<size_t>(unit) * sc.stride + (row - unit * sc.tokens);
}

}  // namespace q4
}  // namespace kvc
