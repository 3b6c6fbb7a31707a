// gdn_recurrence.cuh -- the gates of the gated linear recurrence (include/gdn.h),
// on pairs of channels.
//
//   t = e^-|z|, softplus(z) = max(z, 0) + log1p(t), g = -E softplus(z), alpha = e^g
//   w = 1 - alpha^2 = -expm1(2g), s = sqrt(w), beta = 1 / (1 + e^-b)
//
// Long memory lives where softplus(z) is small and alpha close to 1, so neither
// log(1 + t) nor 1 - alpha^2 may be taken literally: log1p(t) / t on [0, 1] and
// -expm1(-y) / y on [0, 1/2] are polynomials fitted here (weighted least squares to
// the minimax relative error at Chebyshev nodes: 1.4e-7 and 5e-8 with fp32
// evaluation). They run on the fp32 pipe as register pairs, which leaves five
// special-function results per element (three e^x, one reciprocal, one root).
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2_pair(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_pair(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }

// log(1 + t) for t in [0, 1]
__device__ __forceinline__ float2 log1p_unit(float2 t) {
    float2 p = splat2(0.005232691299170256f);
    p = fma2(p, t, splat2(-0.029505228623747826f));
    p = fma2(p, t, splat2(0.07822593301534653f));
    p = fma2(p, t, splat2(-0.13663244247436523f));
    p = fma2(p, t, splat2(0.19106006622314453f));
    p = fma2(p, t, splat2(-0.2484298199415207f));
    p = fma2(p, t, splat2(0.3331909775733948f));
    p = fma2(p, t, splat2(-0.4999949336051941f));
    p = fma2(p, t, splat2(0.9999999403953552f));
    return mul2(t, p);
}

// 1 - e^-y for y in [0, 1/2]
__device__ __forceinline__ float2 one_minus_exp_small(float2 y) {
    float2 p = splat2(-0.0011216348502784967f);
    p = fma2(p, y, splat2(0.008187386207282543f));
    p = fma2(p, y, splat2(-0.041629090905189514f));
    p = fma2(p, y, splat2(0.16666224598884583f));
    p = fma2(p, y, splat2(-0.4999998211860657f));
    p = fma2(p, y, splat2(1.0f));
    return mul2(y, p);
}

// Decay of two channels from the gate input a. rate = exp(A_log).
struct Decay2 {
    float2 z, t;    // a + dt_bias, e^-|z|
    float2 sp;      // softplus(z)
    float2 alpha;   // e^-(rate sp)
    float2 w;       // 1 - alpha^2
};

__device__ __forceinline__ Decay2 decay2(float2 a, float2 bias, float2 rate) {
    Decay2 r;
    r.z = add2(a, bias);
    r.t = ex2_pair(make_float2(-fabsf(r.z.x) * kLog2e, -fabsf(r.z.y) * kLog2e));
    r.sp = add2(make_float2(fmaxf(r.z.x, 0.f), fmaxf(r.z.y, 0.f)), log1p_unit(r.t));
    const float2 y = mul2(rate, r.sp);   // -log(alpha)
    // alpha = 1 - em with em = 1 - e^-y from the polynomial where y < 1/2 (the long memories: the
    // hardware exponential's last bits would pile up over thousands of tokens), else e^-y
    const float2 es = one_minus_exp_small(y);
    const float2 al = ex2_pair(mul2(y, splat2(-kLog2e)));
    const float2 el = fma2(al, splat2(-1.f), splat2(1.f)), as = fma2(es, splat2(-1.f), splat2(1.f));
    const float2 em = make_float2(y.x < 0.5f ? es.x : el.x, y.y < 0.5f ? es.y : el.y);
    r.alpha = make_float2(y.x < 0.5f ? as.x : al.x, y.y < 0.5f ? as.y : al.y);
    r.w = fma2(em, r.alpha, em);
    return r;
}

// 1 / sqrt(w) for the scale s = w / sqrt(w); a w below the normal range (where the
// approximation flushes) gives s = 0, a NaN stays one through w.
__device__ __forceinline__ float2 inv_sqrt2(float2 w) {
    return make_float2(rsqrt_approx(fmaxf(w.x, 1.17549435e-38f)), rsqrt_approx(fmaxf(w.y, 1.17549435e-38f)));
}

__device__ __forceinline__ float2 sigmoid2(float2 b) {
    return rcp_pair(add2(ex2_pair(mul2(b, splat2(-kLog2e))), splat2(1.f)));
}

// sigmoid(z) from t = e^-|z|
__device__ __forceinline__ float2 sigmoid_from_t(float2 z, float2 t) {
    const float2 r = rcp_pair(add2(t, splat2(1.f)));
    const float2 q = mul2(t, r);
    return make_float2(z.x >= 0.f ? r.x : q.x, z.y >= 0.f ? r.y : q.y);
}

}  // namespace gdn
