// pa_fp4.cuh - the 4-bit pool: where a row lies, and how elements become codes and back.
//
// A pool is uint8 [num_blocks][num_kv_heads][2][tile]: K, then V, of one (block, head), each
// tile = block_size rows of head_size / 2 bytes (element 2i is the low nibble of byte i, an OCP
// e2m1 code), then block_size rows of head_size / 16 e4m3 scales, one per 16 elements.  An
// element is code * scale * g, g the tensor's k_scale or v_scale.  K and V of a (block, head)
// are one run of block_size * head_size * 9 / 8 bytes.
#pragma once

#include <cmath>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kFp4Group = 16;  // elements that share a scale

struct Fp4Row {
    int64_t codes, scale;  // byte offsets of a row's codes and of its scales
};

template <int D>
__device__ __forceinline__ Fp4Row fp4_row(int blk, int off, int head, int side, int num_kv_heads,
                                          int block_size) {
    const int tile = block_size * (D * 9 / 16);
    const int64_t base = (((int64_t)blk * num_kv_heads + head) * 2 + side) * tile;
    return {base + off * (D / 2), base + block_size * (D / 2) + off * (D / 16)};
}

// Eight fp32 values to e2m1 codes (nearest, ties to the even code, saturating at 6), the first
// in the lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight e2m1 codes (the nibbles of w, lowest first) to four f16x2 words, exactly.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// Two e4m3 codes (the low bytes of w) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// max(|a|, |b|) of bf16 pairs, NaN if either is.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
}

// Quotients by d without dividing.  With r within 2^-23 of 1 / d (relatively), x r (1 - 2^-20)
// and x r (1 + 2^-20) lie on both sides of the quotient x / d and of its rounding to binary32 (off
// by 2^-23, and by 2^-24 for each of r's factor, the product and the quotient: five of sixteen
// 2^-24), and a code does not fall as its value's magnitude rises: where both products give one
// code it is the quotient's.  The rest, next to a tie, is divided.
struct Around {
    float lo, hi;  // r (1 - 2^-20), r (1 + 2^-20); 0 where 1 / d or the products may not be normal
};

// Of a positive divisor known on the host.
inline Around around(float d) {
    if (!(d > 1e-30f && d < 1e30f)) return {0.f, 0.f};
    int e;
    if (std::frexp(d, &e) == 0.5f) return {1.f / d, 1.f / d};  // a power of two: exact
    return {(float)((1.0 - 0x1p-20) / d), (float)((1.0 + 0x1p-20) / d)};
}

// Eight bf16 elements over d as e4m3 codes (nearest, ties to even, saturating).
__device__ __forceinline__ uint2 e4m3_of_quotients(const uint4 &x, float d, const Around &r) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float v[4], lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            lo[i] = hi[i] = v[i] = bf16_lo(w[2 * k + i / 2]);
            lo[i + 1] = hi[i + 1] = v[i + 1] = bf16_hi(w[2 * k + i / 2]);
            mul2(lo[i], lo[i + 1], r.lo, r.lo);
            mul2(hi[i], hi[i + 1], r.hi, r.hi);
        }
        c[k] = pack_e4m3x2(lo[0], lo[1]) | pack_e4m3x2(lo[2], lo[3]) << 16;
        if (r.lo == 0.f ||
            c[k] != (pack_e4m3x2(hi[0], hi[1]) | pack_e4m3x2(hi[2], hi[3]) << 16))
            c[k] = pack_e4m3x2(__fdiv_rn(v[0], d), __fdiv_rn(v[1], d)) |
                   pack_e4m3x2(__fdiv_rn(v[2], d), __fdiv_rn(v[3], d)) << 16;
    }
    return make_uint2(c[0], c[1]);
}

// A tensor's scale g, h = fp32(6 g), and what divides by h.
struct Fp4Scale {
    float g, h;
    Around by_h;
};
inline Fp4Scale fp4_scale(float g) { return {g, 6.f * g, around(6.f * g)}; }

// Sixteen bf16 elements (x[0] holds the first two) to their scale's e4m3 code (returned) and
// e2m1 codes:  s = e4m3(max|x| / h);  d = fp32(s g);  code = e2m1(x / d), all divisions
// binary32's, roundings to nearest even, saturating.  A group whose d is not above 0 (max|x| too
// small for a scale, or a NaN) has codes of 0; with a NaN its scale is NaN too, so that all its
// elements are.  (A division per element took 390 instructions for a warp's 32 groups; this
// takes some 190.)
__device__ __forceinline__ uint32_t fp4_quantise(const uint32_t (&x)[8], const Fp4Scale &t,
                                                 uint2 &codes) {
    uint32_t m = absmax_bf16x2(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) m = absmax_bf16x2(m, x[i]);
    m = absmax_bf16x2(m, m >> 16);
    const float top = bf16_lo(m);
    uint32_t s = pack_e4m3x2(top * t.by_h.lo, top * t.by_h.hi);
    if (t.by_h.lo == 0.f || (s & 0xffu) != s >> 8) s = pack_e4m3x2(__fdiv_rn(top, t.h), 0.f);
    s &= 0xffu;
    const float d = __fmul_rn(f16_lo(e4m3x2_to_f16x2(s)), t.g);
    codes = make_uint2(0u, 0u);
    if (!(d > 0.f)) return s;
    const bool tame = d > 1e-30f && d < 1e30f;
    // With a d of at most 12 bits (any s, g a power of two) ties are common, and nothing else is
    // near one: x has 8 bits, the middle between two codes 3, so a quotient that is not the
    // middle is off it by 2^-15 at least.  There one product is enough, rounded to 18 bits, which
    // takes a tie's error (below 2^-22) away and moves no other across.
    const bool few_bits = (__float_as_uint(d) & 0xfffu) == 0u;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float r0 = r * (1.f - 0x1p-20f), r1 = r * (1.f + 0x1p-20f);
    uint32_t c[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float v[8], lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            v[i] = bf16_lo(x[4 * w + i / 2]);
            v[i + 1] = bf16_hi(x[4 * w + i / 2]);
        }
        if (tame && few_bits) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                mul2(v[i], v[i + 1], r, r);
                v[i] = __uint_as_float((__float_as_uint(v[i]) + 0x20u) & ~0x3fu);
                v[i + 1] = __uint_as_float((__float_as_uint(v[i + 1]) + 0x20u) & ~0x3fu);
            }
            c[w] = pack_e2m1x8(v);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            lo[i] = hi[i] = v[i];
            lo[i + 1] = hi[i + 1] = v[i + 1];
            mul2(lo[i], lo[i + 1], r0, r0);
            mul2(hi[i], hi[i + 1], r1, r1);
        }
        c[w] = pack_e2m1x8(lo);
        if (!tame || c[w] != pack_e2m1x8(hi)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], d);
            c[w] = pack_e2m1x8(v);
        }
    }
    codes = make_uint2(c[0], c[1]);
    return s;
}

// 32 bytes at once (p 32-byte aligned).
__device__ __forceinline__ void ld_32(uint32_t (&v)[8], const void *p) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void st_32(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

}  // namespace pa
