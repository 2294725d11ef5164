// scoremod.cuh -- the tanh cap of modified scores, shared by the forward and the backward kernels.
//
// tanh(u) = u P(u^2) with a polynomial fitted to tanh(u) / u over |u| <= 1 (iterated weighted least
// squares: relative error 6e-7, 7e-7 with the roundings of fp32): eight packed operations per two
// scores and no special-function unit.  Scores with a larger |u| take the exponential form 1 - 2 / (1 +
// e^(2|u|)), whose cancellation is harmless from |u| = 1 on; a warp takes it as one, and only where one
// of its scores needs it.
#pragma once

#include "sm103_ptx.cuh"

namespace attn {

// tanh(u) for u >= 1 (1 once e^(2u) overflows).
__device__ __forceinline__ float tanh_large(float u) {
    return 1.f - __fdividef(2.f, 1.f + ex2_approx(u * 2.885390082f));  // 2 log2(e)
}

struct TanhPoly {
    uint64_t a[6];   // coefficients times `out`, as packed pairs
    float out;
    __device__ __forceinline__ explicit TanhPoly(float out_) : out(out_) {
        constexpr float kP[6] = {0.999999414f, -0.333290424f, 0.13281434f, -0.0516056762f, 0.0167431162f, -0.00306706033f};
#pragma unroll
        for (int i = 0; i < 6; ++i) a[i] = f32x2_pack(kP[i] * out, kP[i] * out);
    }
    // out * tanh of a packed pair; far: some |u| of the warp may exceed 1
    __device__ __forceinline__ uint64_t operator()(uint64_t u, bool far) const {
        const uint64_t z = f32x2_mul(u, u);
        uint64_t t = f32x2_fma(z, a[5], a[4]);
#pragma unroll
        for (int k = 3; k >= 0; --k) t = f32x2_fma(z, t, a[k]);
        t = f32x2_mul(t, u);
        if (far) {
            float u0, u1, t0, t1;
            f32x2_unpack(u, u0, u1);
            f32x2_unpack(t, t0, t1);
            t0 = fabsf(u0) > 1.f ? copysignf(tanh_large(fabsf(u0)) * out, u0) : t0;
            t1 = fabsf(u1) > 1.f ? copysignf(tanh_large(fabsf(u1)) * out, u1) : t1;
            t = f32x2_pack(t0, t1);
        }
        return t;
    }
};

// Largest |x| of the scores a thread holds.
template <int H>
__device__ __forceinline__ float abs_max(const uint32_t (&s)[H][32]) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < 32; ++i) m[i & 3] = fmaxf(m[i & 3], fabsf(__uint_as_float(s[h][i])));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

}  // namespace attn
