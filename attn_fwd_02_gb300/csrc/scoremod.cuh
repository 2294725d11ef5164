// scoremod.cuh -- the tanh cap of modified scores, shared by the forward, backward and decode kernels.
//
// out * tanh(u), u = in * raw, without the special-function unit where the scores allow it:
//   near  |u| <= 1/4:  raw P3(raw^2), a polynomial of three terms whose coefficients carry in and out
//                      (relative error 5e-7): four FMA-pipe operations a score;
//   mid   |u| <= 1:    u P6(u^2), six terms (7e-7): eight operations;
//   far                the exponential form 1 - 2 / (1 + e^(2|u|)) where |u| > 1 (its cancellation is
//                      harmless from there on), the six terms elsewhere.
// The polynomials are fits of tanh(u) / u in u^2 by iterated weighted least squares.  A warp takes the
// tier that its largest |u| needs, as one: one score past the cap sends all of a warp's through the exponential form.
// Measured on a causal forward / backward of 16 heads x 8192, us, with no cap and with the largest score at 0.2, 0.7,
// 1.5 and 4 times the cap: d = 128 249 / 929, 316 / 1043, 396 / 1080, 807 / 1109, 665 / 1306; d = 64 171 / 718, 258 / 879,
// 335 / 967, 344 / 973, 516 / 1216.
#pragma once

#include "sm103_ptx.cuh"

namespace attn {

__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// tanh(u) for u >= 1 (1 once e^(2u) overflows).
__device__ __forceinline__ float tanh_large(float u) {
    return 1.f - __fdividef(2.f, 1.f + ex2_approx(u * 2.885390082f));  // 2 log2(e)
}

struct TanhCap {
    float in, out;
    uint64_t n0, n1, n2;  // near coefficients, as packed pairs
    bool near_ok;         // they are all well inside the normal range of fp32

    __device__ __forceinline__ TanhCap(float in_, float out_) : in(in_), out(out_) {
        const float a = in * out, s = in * in;
        n0 = f32x2_pack(0.999999604f * a, 0.999999604f * a);
        n1 = f32x2_pack(-0.333219082f * a * s, -0.333219082f * a * s);
        n2 = f32x2_pack(0.128416134f * a * s * s, 0.128416134f * a * s * s);
        const float most = fmaxf(a, a * s * s), least = fminf(a, a * s * s);
        near_ok = most < 1e36f && least > 1e-36f;
    }
    // 0 near, 1 mid, 2 far for a warp whose lanes hold scores up to `big` in absolute value.
    __device__ __forceinline__ int tier(float big) const {
        const float u = big * in;
        if (near_ok && !__any_sync(0xffffffffu, u > 0.25f)) return 0;
        return __any_sync(0xffffffffu, u > 1.f) ? 2 : 1;
    }
    template <int T>
    __device__ __forceinline__ uint64_t eval(uint64_t raw) const {
        if constexpr (T == 0) {
            const uint64_t z = f32x2_mul(raw, raw);
            return f32x2_mul(f32x2_fma(z, f32x2_fma(z, n2, n1), n0), raw);
        } else {
            return eval_u<T>(f32x2_mul(raw, f32x2_pack(in, in)), out);
        }
    }
    // out * tanh(u) of a pair, by the mid (1) or the far (2) form.
    template <int T>
    static __device__ __forceinline__ uint64_t eval_u(uint64_t u, float out) {
        constexpr float kP[6] = {0.999999414f, -0.333290424f, 0.13281434f,
                                 -0.0516056762f, 0.0167431162f, -0.00306706033f};
        const uint64_t z = f32x2_mul(u, u);
        uint64_t t = f32x2_fma(z, f32x2_pack(kP[5] * out, kP[5] * out), f32x2_pack(kP[4] * out, kP[4] * out));
#pragma unroll
        for (int k = 3; k >= 0; --k) t = f32x2_fma(z, t, f32x2_pack(kP[k] * out, kP[k] * out));
        t = f32x2_mul(t, u);
        if constexpr (T == 2) {
            float u0, u1, t0, t1;
            f32x2_unpack(u, u0, u1);
            f32x2_unpack(t, t0, t1);
            t0 = fabsf(u0) > 1.f ? copysignf(tanh_large(fabsf(u0)) * out, u0) : t0;
            t1 = fabsf(u1) > 1.f ? copysignf(tanh_large(fabsf(u1)) * out, u1) : t1;
            t = f32x2_pack(t0, t1);
        }
        return t;
    }
    // One score.
    __device__ __forceinline__ float one(int tier, float raw) const {
        const uint64_t r = f32x2_pack(raw, raw);
        float a, b;
        f32x2_unpack(tier == 0 ? eval<0>(r) : (tier == 1 ? eval<1>(r) : eval<2>(r)), a, b);
        return a;
    }
    // A thread's scores, in place.
    template <int T, int H>
    __device__ __forceinline__ void apply_tier(uint32_t (&s)[H][32]) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float a, b;
                f32x2_unpack(eval<T>(f32x2_pack(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 1]))), a, b);
                s[h][i] = __float_as_uint(a);
                s[h][i + 1] = __float_as_uint(b);
            }
    }
    template <int H>
    __device__ __forceinline__ void apply(int tier, uint32_t (&s)[H][32]) const {
        if (tier == 0) apply_tier<0, H>(s);
        else if (tier == 1) apply_tier<1, H>(s);
        else apply_tier<2, H>(s);
    }
};

// A slope in the log2 domain; finite whatever the slope, so that a distance of 0 adds 0.
__device__ __forceinline__ float bias_slope(float slope) {
    return fminf(fmaxf(slope * 1.4426950408889634f, -3.4028235e38f), 3.4028235e38f);
}
// Up to this slope (log2 domain) the forward takes the bias of a tile as linear in the column, which is off by 2^-24
// of its largest value in the tile, 128 slopes (3e-5 of a score here), where -slope |distance| is off by 2^-24 of
// itself: a steep slope's error would swamp the keys near the query, whose weights are the ones left.
constexpr float kLinearSlope = 4.f;

// Smallest of the 64 scores a thread holds (four chains of three-input minima).
__device__ __forceinline__ float min64(const uint32_t (&s)[2][32]) {
    float m[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) m[a] = fminf(__uint_as_float(s[0][a]), __uint_as_float(s[1][a]));
#pragma unroll
    for (int i = 4; i < 32; i += 4)
#pragma unroll
        for (int a = 0; a < 4; ++a) m[a] = fmin3(m[a], __uint_as_float(s[0][i + a]), __uint_as_float(s[1][i + a]));
    return fminf(fminf(m[0], m[1]), fminf(m[2], m[3]));
}
// Largest absolute value of a thread's scores.
template <int H>
__device__ __forceinline__ float abs_max(const uint32_t (&s)[H][32]) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int a = 0; a < 4; ++a) m[a] = fmax3_abs(m[a], __uint_as_float(s[h][i + 2 * a]), __uint_as_float(s[h][i + 2 * a + 1]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// Largest of them.
__device__ __forceinline__ float max64_of(const uint32_t (&s)[2][32]) {
    float m[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) m[a] = fmaxf(__uint_as_float(s[0][a]), __uint_as_float(s[1][a]));
#pragma unroll
    for (int i = 4; i < 32; i += 4)
#pragma unroll
        for (int a = 0; a < 4; ++a) m[a] = fmax3(m[a], __uint_as_float(s[0][i + a]), __uint_as_float(s[1][i + a]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

}  // namespace attn
