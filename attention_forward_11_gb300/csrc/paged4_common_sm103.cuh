// paged4_common_sm103.cuh -- what the attention kernels over a cache in 4 bits share.
//
// A cached element is code x scale x unit: an e2m1 code (two to a byte, the first in the low
// half), the e4m3 scale of its block of 16, and one number for the cache.  code x scale has at
// most 6 significant bits and, scales from 2^-9 to 448, lies in [2^-10, 2688]: exact in fp16.  So
// K and V become fp16 operands without rounding, by one conversion and one product for two
// elements, whatever q's type; the units go into the softmax scale and into O.  bf16 queries
// become fp16 too: a row is scaled by a power of two that brings its largest element to
// [2^14, 2^15), exactly but for elements below 2^-28 of that (off by at most 2^-39 of it), and
// its logits are scaled back.
#pragma once
#include <cfloat>
#include <cstdint>

#include "paged_common_sm103.cuh"

namespace attn {
namespace paged {

// Weights are 2^(exponent - m) for an m that is kMaxBelow below the row's maximum when it is set and is set anew
// when the maximum is past it by more than kMaxAbove, so all are at most 2^15 and fp16 holds them.  Weights of the
// keys far below the maximum are fp16's small numbers, of steps of 2^-24: 2^-31 of the largest, where an m at the
// maximum itself would lose all that 10^6 keys at 2^-26 of it sum to, a 60th of O.
constexpr float kMaxBelow = 7.f, kMaxAbove = 15.f;

// An exponent is one fused product, whose product is exact, less an m that was rounded: off by up to half a step of
// m, in all of a row's weights alike.  Below 2^23 that is at most 1/2, and weights stay below fp16's 65504; the
// entry point's contract ends there.

struct Paged4Params : PagedParams {  // its strides are the codes', in bytes
    const uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
    long long scale_page, scale_token, scale_head;  // bytes
    float v_unit;  // k's is part of scale_log2
    int f16;       // q's and o's type
};

// four bytes of two codes each -> four pairs of fp16, the low half's code in the low half
__device__ __forceinline__ void e2m1_to_f16(uint32_t (&h)[4], uint32_t w) {
    asm("{.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// two e4m3 in the low half of `two` -> a pair of fp16
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}
__device__ __forceinline__ uint32_t low_twice(uint32_t h) { return __byte_perm(h, 0, 0x1010); }
__device__ __forceinline__ uint32_t high_twice(uint32_t h) { return __byte_perm(h, 0, 0x3232); }

// The power of two that a row of bf16 is multiplied by to become fp16, from the largest bits of
// its sizes, and its inverse: 2^14 over the power of two below the largest element, kept where
// both are normal numbers (of an infinite row: 2^-114, which leaves infinities as they are).
__device__ __forceinline__ float row_factor(uint32_t top_bits, float& inverse) {
    const uint32_t field = min(268u - (top_bits >> 7), 253u);
    inverse = __uint_as_float((254u - field) << 23);
    return __uint_as_float(field << 23);
}
// The scale of such a row's logits: kept a normal number.  A row of zeros, or one whose scale lies below, has
// products of at most 2^35 and so logits of (nearly) zero whatever its scale, but a scale of zero would make NaN
// of a masked logit, and an infinite one of a product of zero.
__device__ __forceinline__ float row_scale(float scale_log2, float inverse) {
    return fminf(fmaxf(scale_log2 * inverse, FLT_MIN), FLT_MAX);
}
// two bf16 times a factor -> two fp16
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x, float factor) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
        : "=r"(h)
        : "f"(__uint_as_float(x & 0xffff0000u) * factor), "f"(__uint_as_float(x << 16) * factor));
    return h;
}

}  // namespace paged
}  // namespace attn
