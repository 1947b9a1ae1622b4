// q8_format.cuh -- the 8-bit checkpoint format: encoding and decoding of one
// block of 32 consecutive columns of a row.
//
// A block shares one exponent byte E, the power-of-two scale of the OCP
// microscaling formats (E8M0, blocks of 32):
//
//   INT8  value = code * 2^(E - 133)    code a two's complement byte, -127 .. 127
//   E4M3  value = code * 2^(E - 127)    code an 8-bit float, 4 exponent and 3
//                                       mantissa bits, largest magnitude 448
//
// E is the smallest exponent at which the block's largest magnitude amax is
// representable without saturation (amax <= 127 * 2^(E-133), respectively
// amax <= 448 * 2^(E-127)).  That comparison is an integer addition to the
// float's bits: 127 = 1.984375 * 2^6, so adding the distance of mantissa
// 0x7E0000 from the next binade carries into the exponent exactly when amax
// is above it (448 = 1.75 * 2^8, mantissa 0x600000, likewise).  E is clamped
// from below so that every nonzero value is a normal fp32 number (7 and 10),
// and for INT8 from above at 254 (there 127 * 2^121 is the nearest value to
// what lies above it).  A power of two scales exactly, so the only rounding
// is the one to the code (to nearest, ties to even), and every value has at
// most 7 significant bits: it is exactly a bf16 number, which is how the
// tensor-core product reads it.  (E4M3 under E = 247 rounds to nearest beyond
// the largest float: 248 * 2^120 and more, to 2^128, which reads as infinity.)
//
// E = 255 marks a block that holds a NaN or an infinity: its codes are 0 and
// every element of it restores to NaN, so that an overflow in the forward
// pass is seen in the gradients.  Bytes the encoder does not produce: E below
// the clamp reads as a scale of zero.
#pragma once

#include <cstdint>

namespace gemm_f32_dev {

constexpr int kQ8Int8 = 0;
constexpr int kQ8E4m3 = 1;
constexpr int kQ8Block = 32;

constexpr unsigned kQ8NonFinite = 255u;

// Exponent byte of a block from the bits of its largest magnitude (as an
// unsigned maximum of the values' bits without sign: a NaN is the largest).
template <int FMT>
__device__ __forceinline__ unsigned q8_exponent(unsigned amax_bits) {
    unsigned e;
    if (FMT == kQ8Int8)
        e = min(254u, max(7u, (amax_bits + 0x1FFFFu) >> 23));
    else
        e = max(18u, (amax_bits + 0x1FFFFFu) >> 23) - 8u;
    return amax_bits >= 0x7F800000u ? kQ8NonFinite : e;
}

// 2^-(scale exponent): what a value is multiplied with before rounding.
template <int FMT>
__device__ __forceinline__ float q8_inverse_scale(unsigned e) {
    return __uint_as_float(((FMT == kQ8Int8 ? 260u : 254u) - e) << 23);
}

// The scale of exponent byte e as a float: NaN for 255, 0 below the clamp.
template <int FMT>
__device__ __forceinline__ float q8_scale(unsigned e) {
    const unsigned field = FMT == kQ8Int8 ? e - 6u : e;
    const unsigned bits = e == kQ8NonFinite ? 0x7FFFFFFFu
                          : e < (FMT == kQ8Int8 ? 7u : 10u) ? 0u : field << 23;
    return __uint_as_float(bits);
}

// Codes of four values (inv = q8_inverse_scale(e)), value 0 in the low byte.
// INT8: adding 1.5 * 2^23 leaves the integer nearest to the value (ties to
// even) in the low bits of the sum, and as the product with a power of two
// is exact one fused multiply-add rounds alike.  Only where E is held at 254
// can a value round to 128, and be clamped.
template <int FMT>
__device__ __forceinline__ unsigned q8_encode4(float a, float b, float c, float d, float inv,
                                               unsigned e) {
    unsigned w;
    if (FMT == kQ8Int8) {
        const float magic = 12582912.0f;
        if (e >= 254u) {
            const float top = 127.0f * __uint_as_float((e - 6u) << 23);  // 127 * 2^121
            a = fminf(fmaxf(a, -top), top);
            b = fminf(fmaxf(b, -top), top);
            c = fminf(fmaxf(c, -top), top);
            d = fminf(fmaxf(d, -top), top);
        }
        const unsigned qa = __float_as_uint(fmaf(a, inv, magic));
        const unsigned qb = __float_as_uint(fmaf(b, inv, magic));
        const unsigned qc = __float_as_uint(fmaf(c, inv, magic));
        const unsigned qd = __float_as_uint(fmaf(d, inv, magic));
        w = __byte_perm(__byte_perm(qa, qb, 0x0040), __byte_perm(qc, qd, 0x0040), 0x5410);
    } else {
        unsigned short lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
        w = static_cast<unsigned>(lo) | (static_cast<unsigned>(hi) << 16);
    }
    return e == kQ8NonFinite ? 0u : w;
}

// The four numbers of a code word, unscaled.
template <int FMT>
__device__ __forceinline__ float4 q8_decode4(unsigned w) {
    if (FMT == kQ8Int8) {
        // byte b of w with its sign bit flipped is code + 128, placed in the
        // low mantissa bits of 2^23
        const unsigned u = w ^ 0x80808080u;
        const float bias = 8388736.0f;  // 2^23 + 128
        return make_float4(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - bias,
                           __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - bias,
                           __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - bias,
                           __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - bias);
    }
    unsigned lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<unsigned short>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<unsigned short>(w >> 16)));
    float4 v;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v.z), "=f"(v.w)
        : "r"(hi));
    return v;
}

// Bits of |x|, for the unsigned maximum.
__device__ __forceinline__ unsigned q8_magnitude(float x) {
    return __float_as_uint(x) & 0x7FFFFFFFu;
}

}  // namespace gemm_f32_dev
