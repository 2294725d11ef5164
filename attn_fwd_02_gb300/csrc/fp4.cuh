// fp4.cuh -- pages of the 4-bit cache.
//
// A value is e2m1(code) * e4m3(scale) * the tensor's fp32 scale: 4-bit codes (a sign, two exponent bits of bias 1, one
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one e4m3 scale per block of 16 dims of a token, 4.5 bits a value.  A
// product of code and block scale has at most 6 significant bits and lies in f16's normal range (or is 0), so it is exact
// in f16.
//
// One page of one head is 9 d contiguous bytes: 8 d of codes, then d of block scales, ordered for the fragments of the
// decode kernel's products:
//   keys    codes [16 tokens][d / 2]: byte x holds dims 2x (low nibble) and 2x + 1; scales [16 tokens][d / 16].  The
//           products sum over the dims, of which a lane takes neighbours.
//   values  codes [d / 16 blocks][4 quads][2][16 dims]: byte (q, h, x) of a block holds dim x of tokens 2q + 8h (low
//           nibble) and 2q + 8h + 1; scales [4 quads][d / 16][2][2].  The products sum over the tokens, so a byte widens
//           to the pair of tokens that one operand register holds, and a block is one 8 x 8 matrix of ldmatrix.
#pragma once

#include <cuda_fp8.h>

#include "sm103_ptx.cuh"

namespace attn {

constexpr int kFp4PS = 16;  // tokens of a page

// Where a byte lies in a page's block.  Keys: the 8 codes' bytes of 16-dim block j of a token, and their scale.
__host__ __device__ constexpr int fp4_k_codes(int d, int token, int j) { return token * (d / 2) + 8 * j; }
__host__ __device__ constexpr int fp4_k_scale(int d, int token, int j) { return 8 * d + token * (d / 16) + j; }
// Values: the 16 bytes of block j of the token's pair, and the token's scale.
__host__ __device__ constexpr int fp4_v_codes(int token, int j) {
    return j * 128 + ((token & 7) >> 1) * 32 + (token >> 3) * 16;
}
__host__ __device__ constexpr int fp4_v_scale(int d, int token, int j) {
    return 8 * d + ((token & 7) >> 1) * (d / 4) + j * 4 + (token >> 3) * 2 + (token & 1);
}

// Both halves of a word: the f16 value of byte `i` of e4m3 codes.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

// Eight e2m1 codes -> four f16x2 words: r[i] holds the codes of byte i, the low nibble in the low half.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Eight fp32 values -> e2m1 codes, nearest (ties to even), saturating at 6; f[0] in the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&f)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
    uint32_t h;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(code & 0xffu));
    float f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

// A block of 16 values u (already times 1 / the tensor's scale), in place of which it leaves the quotients by the block's scale
// s = e4m3(max |u| / 6), nearest and at most 448, with 1/6 as an fp32 factor; returns the scale's code.
//
// The quotients are correctly rounded, so that a code is a function of the definition alone: with r the nearest to 1 / s, q = u r
// and the remainder u - q s (exact by fused multiply-add), q + remainder * r is the nearest to u / s (Markstein's theorem, IBM J.
// Res. Dev. 34 (1990)), two at a time in packed arithmetic.  Values past 2^100 times the tensor's scale, all of whose quotients
// are far above the largest code or lost below it, are cut to that first.  Of a block with scale 0 the quotients are any; its
// codes are to be 0.
__device__ __forceinline__ uint32_t fp4_quotients(float (&u)[16]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) m = fmaxf(m, fmaxf(fabsf(u[i]), fabsf(u[i + 1])));
    constexpr float kMost = 1.2676506e30f;  // 2^100
    if (m > kMost) {
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = fminf(fmaxf(u[i], -kMost), kMost);
    }
    const uint32_t code = __nv_cvt_float_to_fp8(__fmul_rn(m, 0.16666667163372039794921875f), __NV_SATFINITE, __NV_E4M3);
    const float s = e4m3_to_float(code), r = s > 0.f ? __frcp_rn(s) : 0.f;
    const uint64_t r2 = f32x2_pack(r, r), s2 = f32x2_pack(-s, -s);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const uint64_t x = f32x2_pack(u[i], u[i + 1]), q = f32x2_mul(x, r2);
        float y0, y1;
        f32x2_unpack(f32x2_fma(f32x2_fma(q, s2, x), r2, q), y0, y1);
        u[i] = copysignf(y0, u[i]);  // (-0 stays -0)
        u[i + 1] = copysignf(y1, u[i + 1]);
    }
    return code;
}

}  // namespace attn
