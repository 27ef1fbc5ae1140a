// paged4_append_sm103.cuh -- keys and values written into a paged cache in 4 bits.
//
// A row of D elements is cut into blocks of 16.  With y = x / unit (one fp32 product with
// 1 / unit) a block's scale is s = e4m3(max |y| / 6), rounded to nearest even, at most 448
// and at least 2^-9 unless the block is zero, and an element's code is e2m1(y / s), rounded
// to nearest with ties to the even code, 6 for all above.  Both roundings are exact: the
// quotient that cvt rounds is y r (r = 1 / s) corrected by its remainder, y r + (y - (y r) s) r
// with two fused products, which is within half a unit of its last place of y / s and equal to
// it where y / s has few bits, as every border between two codes has (without the correction
// 11 of the 56 pairs of a significand and a border fall on the wrong side).  Where the unit is a
// power of two, y has as few bits as x: a quotient that is no border is at least 2^-12 of itself
// away from one, the products y r that miss a border are one last place above it, and
// clearing the product's last 8 bits puts both right (kShort: 3 instructions an element, not 6).
// A NaN or an infinity makes its block's scale 448 and is stored as +-6 (a NaN as +6).
//
// A thread has one block of K and the same block of V: 64 bytes read, 16 bytes of codes and
// two bytes of scales written, four lanes' scales in one word.  65000 rows of 16 heads of 64 in scattered
// slots take 74 us on pages stored head by head (78 without kShort), 64 token by token (5.3 TB/s); 64 rows of
// 8 heads 2.1 us.  Counters with kShort, head by head / token by token: 62 / 68 % of the issue slots, 58 / 62 %
// of DRAM's rate, half of a warp's time waits for loads.  What stored head by head costs is its writes: a word
// of scales is a sector of its own, 6.3 instead of 3.5 million sectors.
#pragma once
#include <cfloat>
#include <cstdint>

#include "paged_common_sm103.cuh"

namespace attn {
namespace paged {

struct Append4Params {
    const uint16_t *k, *v;  // rows [T, Hkv, D], heads contiguous
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const long long* slot_map;
    long long k_stride, v_stride;                                    // elements from row to row
    long long code_page, code_token, code_head;                      // bytes
    long long scale_page, scale_token, scale_head;
    long long n_slots;
    float k_inv, v_inv;    // 1 / unit
    int T, per_block;      // rows, rows of one block of threads
    int row_blocks;        // blocks of 16 of a row: Hkv * D / 16
    int head_blocks_log2;  // of one head
    FastDiv by_page, by_row;
};

constexpr int kAppend4Threads = 256;

struct Coded {
    uint32_t lo, hi;  // 16 codes
    uint32_t scale;   // e4m3
};

template <bool kF16, bool kShort>
__device__ __forceinline__ Coded encode16(const uint4& a, const uint4& b, float inv) {
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    // the bits of |x| are ordered like |x|, NaN above infinity
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, x[i] & 0x7fff7fffu);
    const uint32_t top_bits = max(top2 & 0xffffu, top2 >> 16);
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (kF16) {
            asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
                : "=f"(y[2 * i]), "=f"(y[2 * i + 1]) : "r"(x[i]));
        } else {
            y[2 * i] = __uint_as_float(x[i] << 16);
            y[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
        if constexpr (!kShort) {
            y[2 * i] *= inv;
            y[2 * i + 1] *= inv;
        }
    }
    float top;
    if constexpr (kF16) asm("{.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(top) : "r"(top_bits));
    else top = __uint_as_float(top_bits << 16);
    top *= inv;
    if (!(top <= FLT_MAX)) {  // a NaN, an infinity, or a unit too small for the row
        top = FLT_MAX;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = fmaxf(fminf(y[i], FLT_MAX), -FLT_MAX);  // kShort: of x, whose quotients saturate
    }
    Coded c;
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(__fdiv_rn(top, 6.f)));
    c.scale = two & 0xffu;
    if (c.scale == 0 && top > 0.f) c.scale = 1;
    uint32_t s2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(static_cast<uint16_t>(c.scale)));
    float s;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(s) : "r"(s2));
    const float r = c.scale == 0 ? 0.f : __frcp_rn(s);
    if constexpr (kShort) {
        const float by = r * inv;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(__float_as_uint(y[i] * by) & 0xffffff00u);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float t = y[i] * r;
            y[i] = copysignf(fmaf(fmaf(-t, s, y[i]), r, t), y[i]);
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm("{.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};}"
            : "=r"(w[i])
            : "f"(y[8 * i]), "f"(y[8 * i + 1]), "f"(y[8 * i + 2]), "f"(y[8 * i + 3]), "f"(y[8 * i + 4]),
              "f"(y[8 * i + 5]), "f"(y[8 * i + 6]), "f"(y[8 * i + 7]));
    c.lo = w[0];
    c.hi = w[1];
    return c;
}

// kShort: both units are powers of two, from 2^-99 to 2^101.
template <bool kF16, bool kShort>
__global__ void __launch_bounds__(kAppend4Threads) paged4_append_kernel(const Append4Params p) {
    launch_dependents();
    wait_for_primary();
    const long long row0 = (long long)blockIdx.x * p.per_block;
    const unsigned int n = static_cast<unsigned int>(min((long long)p.per_block, p.T - row0)) * p.row_blocks;
    for (unsigned int i0 = 0; i0 < n; i0 += kAppend4Threads) {
        const unsigned int i = i0 + threadIdx.x;
        const unsigned int r = static_cast<unsigned int>(p.by_row.quot(i)), b = i - r * p.row_blocks;
        const long long slot = i < n ? p.slot_map[row0 + r] : -1;
        const bool there = slot >= 0 && slot < p.n_slots;  // one answer for the four lanes of a word of scales
        uint4 x[4] = {};
        if (there) {
            const uint4* k = reinterpret_cast<const uint4*>(p.k + (row0 + r) * p.k_stride + b * 16ll);
            const uint4* v = reinterpret_cast<const uint4*>(p.v + (row0 + r) * p.v_stride + b * 16ll);
            x[0] = k[0], x[1] = k[1], x[2] = v[0], x[3] = v[1];
        }
        const Coded ck = encode16<kF16, kShort>(x[0], x[1], p.k_inv), cv = encode16<kF16, kShort>(x[2], x[3], p.v_inv);
        uint32_t sk = ck.scale << (8 * (b & 3)), sv = cv.scale << (8 * (b & 3));
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            sk |= __shfl_xor_sync(0xffffffffu, sk, d);
            sv |= __shfl_xor_sync(0xffffffffu, sv, d);
        }
        if (!there) continue;
        const long long page = (long long)p.by_page.quot(slot), row = slot - page * p.by_page.d;
        const unsigned int head = b >> p.head_blocks_log2, hb = b & ((1u << p.head_blocks_log2) - 1);
        const long long code = page * p.code_page + row * p.code_token + head * p.code_head + hb * 8ll;
        *reinterpret_cast<uint2*>(p.k_codes + code) = make_uint2(ck.lo, ck.hi);
        *reinterpret_cast<uint2*>(p.v_codes + code) = make_uint2(cv.lo, cv.hi);
        if ((b & 3) == 0) {
            const long long scale = page * p.scale_page + row * p.scale_token + head * p.scale_head + hb;
            *reinterpret_cast<uint32_t*>(p.k_scales + scale) = sk;
            *reinterpret_cast<uint32_t*>(p.v_scales + scale) = sv;
        }
    }
}

}  // namespace paged
}  // namespace attn
