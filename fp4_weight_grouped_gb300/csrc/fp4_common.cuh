// Rounding to 4-bit floating point with block scales, shared by the quantiser
// and the epilogue that quantises SwiGLU outputs, so both give the same bits.
//
//   MX  one E8M0 byte per 32: e = floor(log2 amax) - 2 (2 = the exponent of the
//       largest e2m1 magnitude, 6), byte = clamp(e + 127, 0, 252), code =
//       e2m1(x * 2^-e), nearest with ties to the even mantissa, saturating at 6.
//       The factor is a power of two, so only the last step rounds.
//   NV  one E4M3 byte per 16 under an f32 tensor scale g: s = e4m3(min(amax /
//       (6 g), 448)), code = e2m1(x * (1 / (s g))).  A block whose s rounds to 0
//       (or whose 1 / (s g) overflows) becomes zeros.
// A block with an infinity or a NaN gets the format's NaN scale (255, 0x7F)
// and zero codes.  -0 is stored as +0, as the weight formats have it.
#pragma once

#include "device_common.cuh"

namespace moe {

constexpr uint32_t kF32Inf = 0x7F800000u;

// E8M0 byte of a block whose largest magnitude has the f32 bits `amax`.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    if (amax >= kF32Inf) return 255u;
    const int e = static_cast<int>(amax >> 23) - 2;   // a subnormal amax has exponent field 0
    return e < 0 ? 0u : static_cast<uint32_t>(e);
}

// 2^(127 - byte): exact for byte 0..252; 0 for the NaN byte (codes become 0).
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127), a subnormal for byte 0; NaN for 255.
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
    if (byte == 0u) return __uint_as_float(0x00400000u);
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte << 23);
}

// E4M3 byte (non-negative) to f32.
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h2;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(h2) : "r"(byte));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h2));
    return f;
}

// E4M3 scale of a block under tensor scale g (g6 = 6 g): nearest, ties to even.
__device__ __forceinline__ uint32_t nv_scale_byte(uint32_t amax, float g6) {
    if (amax >= kF32Inf) return 0x7Fu;
    const float t = fminf(__fdiv_rn(__uint_as_float(amax), g6), 448.0f);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(t));
    return two & 0xFFu;
}

// 1 / (s g), or 0 where the block becomes zeros.
__device__ __forceinline__ float nv_inverse(uint32_t byte, float g) {
    if (byte == 0u || byte == 0x7Fu) return 0.0f;
    const float r = __fdiv_rn(1.0f, e4m3_value(byte) * g);
    return __float_as_uint(r) >= kF32Inf ? 0.0f : r;
}

// Eight f32 -> eight e2m1 codes, v[0] in the lowest nibble (nearest, ties to
// even, saturating).  cvt puts its first operand in the high nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    // -0 -> +0: keep the sign bit only where a magnitude bit is set.
    const uint32_t mag = w & 0x77777777u;
    return mag | (w & (mag + 0x77777777u) & 0x88888888u);
}

// Eight e2m1 codes (value j in nibble j) -> their values.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
            "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "r"(h[i]));
}

}  // namespace moe
