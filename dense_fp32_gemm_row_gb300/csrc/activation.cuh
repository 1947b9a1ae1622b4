// activation.cuh -- the activations of the gated units, in fp32:
//   silu  act(z) = z / (1 + e^-z)
//   gelu  act(z) = z P(z), P the normal distribution function
#pragma once

namespace gemm_f32_dev {

constexpr int kActSilu = 0;
constexpr int kActGelu = 1;

// The normal distribution function below zero, P(-a) = e^(-a^2/2) F(a), with
// F(a) = erfc(a / sqrt 2) e^(a^2/2) / 2 as a polynomial in t = 1 / (1 + 0.35 a)
// without constant term (the form of Hastings, "Approximations for Digital
// Computers", 1955).  The ten coefficients are a weighted least-squares fit
// made for 0 <= a <= 14.5, refined towards equal relative errors: at most
// 5.1e-8 with these coefficients, 3.3e-7 evaluated in fp32.  P(-a) itself has
// that error and the one of the rounded a^2 / 2, which the exponential makes a
// relative error of its own size: measured on gelu, at most 4.5e-7 for a < 2,
// 5.6e-7 to 4, 1.3e-6 to 8, and 4.2e-6 to 13, where P is below 1e-15.  The
// derivative of gelu needs the same exponential.  (erfcf and expf instead:
// 8192 x 8192 forward 164 us, backward 193, bound by instructions.)
__device__ __forceinline__ void normal(float z, float* p, float* bell) {
    const float a = fabsf(z);
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.35f, a, 1.0f)));
    const float e = expf(-0.5f * a * a);
    float f = 0.0030903539154678583f;
    f = fmaf(f, t, -0.04539582133293152f);
    f = fmaf(f, t, 0.18077702820301056f);
    f = fmaf(f, t, -0.3026995360851288f);
    f = fmaf(f, t, 0.19630774855613708f);
    f = fmaf(f, t, -0.04188587889075279f);
    f = fmaf(f, t, 0.11156046390533447f);
    f = fmaf(f, t, 0.1186375617980957f);
    f = fmaf(f, t, 0.13999271392822266f);
    f = fmaf(f, t, 0.13961537182331085f);
    const float below = f * t * e;
    *p = z < 0.0f ? below : 1.0f - below;
    *bell = e;
}

// act(z) and act'(z) in fp32.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float* value, float* slope) {
    if (ACT == kActSilu) {
        const float s = 1.0f / (1.0f + expf(-z));
        *value = z * s;
        *slope = s * fmaf(z, 1.0f - s, 1.0f);
    } else {
        float p, bell;
        normal(z, &p, &bell);
        *value = z * p;
        *slope = fmaf(z * bell, 0.39894228040143268f, p);
    }
}
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    float value, slope;
    act_both<ACT>(z, &value, &slope);
    return value;
}

}  // namespace gemm_f32_dev
