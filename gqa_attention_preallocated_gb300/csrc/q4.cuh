// The 4-bit row format (KVC_Q4, see kvc.h), shared by every kernel that reads
// or writes it.
//
// A row is one token of one KV head, K and V apart: d codes of 4 bits, eight
// to a 32-bit word (value 2i at bits 4i, value 2i + 1 at bits 16 + 4i), and
// one scale word (bf16 step s in the high 16 bits, zero point z, 0 .. 15, in the
// low 16, of which the lowest 4 count).  A value is s * (c - z).
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
__device__ __forceinline__ int zero_of(uint32_t scale_word) { return static_cast<int>(scale_word & 15u); }

// Code of value e (0 .. 7) of a word.
__device__ __forceinline__ int code_of(uint32_t w, int e) { return (w >> (((e & 1) << 4) + ((e >> 1) << 2))) & 15; }

// Range of eight bf16 values: (max(0, x), max(0, -x)) as a bf16 pair.  The
// maxima propagate NaN, so a NaN or an infinity leaves a range that is not
// finite.  Pairs are joined across lanes with max2.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t range8(const uint32_t (&w)[4]) {
    const uint32_t n = 0x80008000u;
    const uint32_t up = max2(max2(w[0], w[1]), max2(w[2], w[3]));
    const uint32_t dn = max2(max2(w[0] ^ n, w[1] ^ n), max2(w[2] ^ n, w[3] ^ n));
    return max2(0u, max2(__byte_perm(up, dn, 0x5410), __byte_perm(up, dn, 0x7632)));
}

// A row's step, reciprocal and zero point from its range, in the format's
// float32 operations; `plain` is false for a row that is stored as zeros (step
// 0) or as NaN (step NaN).
struct RowScale {
    float inv;
    uint32_t word;
    bool plain;
};
__device__ __forceinline__ RowScale row_scale(uint32_t range) {
    RowScale r;
    const float hi = __uint_as_float(range << 16), neg_lo = __uint_as_float(range & 0xFFFF0000u);
    const float span = __fadd_rn(hi, neg_lo);
    const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(span, 15.f)));
    const bool finite = span <= 3.402823466e38f;
    r.plain = finite && s >= kMinStep;
    r.inv = r.plain ? __frcp_rn(s) : 0.f;
    const uint32_t z = r.plain ? static_cast<uint32_t>(__float2int_rn(__fmul_rn(neg_lo, r.inv))) : 0u;
    r.word = r.plain ? (__float_as_uint(s) | z) : (finite ? 0u : 0x7FC00000u);
    return r;
}

// The code word of eight bf16 values of a row.  c = min(15, rint(x / s) + z):
// the lower bound never acts, since x >= lo and rint is odd and monotonic, and
// the upper one acts on the quotient (15 - z is an integer).  Adding 1.5 * 2^23
// rounds to an integer (ties to even) and leaves it in the low bits, modulo
// 2^16; so four codes are one sum of the four floats' bits, shifted, plus
// z * 0x1111, whose low half is the codes' half word.
__device__ __forceinline__ uint32_t encode8(const uint32_t (&w)[4], const RowScale& r) {
    const uint32_t z = r.word & 0xFFFFu;
    const float top = static_cast<float>(15 - static_cast<int>(z));
    uint32_t even = z * 0x1111u, odd = even;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = fminf(__fmul_rn(__uint_as_float(w[i] << 16), r.inv), top);
        const float b = fminf(__fmul_rn(__uint_as_float(w[i] & 0xFFFF0000u), r.inv), top);
        even += __float_as_uint(__fadd_rn(a, 12582912.f)) << (4 * i);
        odd += __float_as_uint(__fadd_rn(b, 12582912.f)) << (4 * i);
    }
    return r.plain ? __byte_perm(even, odd, 0x5410) : 0u;
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
