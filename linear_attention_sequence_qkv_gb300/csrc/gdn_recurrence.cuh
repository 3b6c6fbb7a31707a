// gdn_recurrence.cuh -- the gates of the gated linear recurrence (include/gdn.h),
// on pairs of channels.
//
//   t = e^-|z|, softplus(z) = max(z, 0) + log1p(t), g = -E softplus(z), alpha = e^g
//   em = 1 - alpha, w = 1 - alpha^2 = em + em alpha, s = sqrt(w), beta = 1 / (1 + e^-b)
//
// Everything is kept in powers of two: z, softplus and -g carry a factor log2(e), so
// the exponentials are the hardware's. Long memory lives where softplus(z) is small
// and alpha close to 1, so neither log(1 + t) nor 1 - alpha may be taken literally:
// log2(1 + t) / t on [0, 1] and (1 - 2^-Y) / Y on [0, 1/4] are polynomials fitted here
// (weighted least squares to the minimax relative error at Chebyshev nodes; 3.5e-7 and
// 1.3e-7 in fp32 evaluation). They run on the fp32 pipe as register pairs, which
// leaves five special-function results per element: three exponentials (32 a clock
// and SM), a reciprocal and a root (16).
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLeastNormal = 1.17549435e-38f;

// The constants of the pair operations. `pin` keeps the longer polynomial's in registers: a pair operation takes no
// literal, and left to itself the compiler moves each constant into place before each use. Where 16-bit loads are
// element by element (two CTAs an SM, registers to spare) that gains (40000 x 3001 bf16 with its gradient 1518 against
// 1669 us); where three CTAs share an SM the registers count for more (65536 x 4096 1803 against 1763 us), and so
// where fp32 elements on their way fill them (3 x 19422 x 1147 994 against 940 us).
struct GateConst {
    float2 sp[8], om[4], log2e, one, neg;
    __device__ __forceinline__ static float2 lit(float v) { return make_float2(v, v); }
    __device__ __forceinline__ static float2 pinned(float v) {
        float2 r;
        asm volatile("mov.f32 %0, %1;" : "=f"(r.x) : "f"(v));
        asm volatile("mov.f32 %0, %1;" : "=f"(r.y) : "f"(v));
        return r;
    }
    __device__ __forceinline__ explicit GateConst(bool pin) {
        const float s[8] = {1.4426947832107544f, -0.7213100790977478f, 0.48006370663642883f, -0.3533948063850403f,
                            0.25600969791412354f, -0.15535184741020203f, 0.06360787153244019f, -0.012319467030465603f};
        const float o[4] = {0.6931471228599548f, -0.24022150039672852f, 0.055404357612133026f, -0.008974975906312466f};
#pragma unroll
        for (int i = 0; i < 8; ++i) sp[i] = pin ? pinned(s[i]) : lit(s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) om[i] = lit(o[i]);
        log2e = lit(kLog2e);
        one = lit(1.f);
        neg = lit(-1.f);
    }
};

__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2_pair(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_pair(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
__device__ __forceinline__ float2 one_minus(const GateConst &k, float2 x) { return fma2(x, k.neg, k.one); }

// Decays of N pairs of channels from the gate input a. Step by step over all pairs: each coefficient is
// then fetched once for all of them.
//   z: (a + dt_bias) log2(e), t: e^-|a + dt_bias|, Y: -log2(alpha) = exp(A_log) softplus(a + dt_bias) log2(e),
//   em: 1 - alpha
// In: z holds a. bias2 = dt_bias log2(e) and rate = exp(A_log) of pair i are bias2[i % M], rate[i % M].
template <int N, int M>
__device__ __forceinline__ void decays(const GateConst &C, float2 (&z)[N], const float2 (&bias2)[M], const float2 (&rate)[M], float2 (&t)[N],
                                       float2 (&Y)[N], float2 (&alpha)[N], float2 (&em)[N]) {
    float2 q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = fma2(z[i], C.log2e, bias2[i % M]);
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = ex2_pair(make_float2(-fabsf(z[i].x), -fabsf(z[i].y)));
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = fma2(C.sp[7], t[i], C.sp[6]);
#pragma unroll
    for (int k = 5; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = fma2(q[i], t[i], C.sp[k]);
#pragma unroll
    for (int i = 0; i < N; ++i)
        Y[i] = mul2(rate[i % M], fma2(q[i], t[i], make_float2(fmaxf(z[i].x, 0.f), fmaxf(z[i].y, 0.f))));
    // alpha = 1 - em, with em from the polynomial for slow decays (the hardware exponential's last bits would
    // pile up over thousands of tokens), and the exponential beyond
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = fma2(C.om[3], Y[i], C.om[2]);
#pragma unroll
    for (int k = 1; k >= 0; --k)
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = fma2(q[i], Y[i], C.om[k]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 es = mul2(q[i], Y[i]), al = ex2_pair(make_float2(-Y[i].x, -Y[i].y));
        const float2 as = one_minus(C, es), el = one_minus(C, al);
        const bool s0 = Y[i].x < 0.25f, s1 = Y[i].y < 0.25f;
        em[i] = make_float2(s0 ? es.x : el.x, s1 ? es.y : el.y);
        alpha[i] = make_float2(s0 ? as.x : al.x, s1 ? as.y : al.y);
    }
}

__device__ __forceinline__ float2 sigmoid2(const GateConst &C, float2 b) {
    const float2 m = mul2(b, C.log2e);
    return rcp_pair(add2(ex2_pair(make_float2(-m.x, -m.y)), C.one));
}
// alpha from em and Y
__device__ __forceinline__ float2 decay_of(float2 em, float2 Y) {
    return make_float2(Y.x < 0.25f ? 1.f - em.x : ex2_approx(-Y.x), Y.y < 0.25f ? 1.f - em.y : ex2_approx(-Y.y));
}
// sqrt(1 - alpha^2) sigmoid(b); a 1 - alpha^2 below the normal range counts as 0
__device__ __forceinline__ float2 write_scale2(const GateConst &C, float2 em, float2 alpha, float2 b) {
    const float2 w = fma2(em, alpha, em);
    return mul2(make_float2(sqrt_approx(w.x), sqrt_approx(w.y)), sigmoid2(C, b));
}
// 1 / sqrt(w), finite for w = 0; a NaN stays one through w
__device__ __forceinline__ float2 inv_sqrt2(float2 w) {
    return make_float2(rsqrt_approx(fmaxf(w.x, kLeastNormal)), rsqrt_approx(fmaxf(w.y, kLeastNormal)));
}

// sigmoid(z) from t = e^-|z|
__device__ __forceinline__ float2 sigmoid_from_t(const GateConst &C, float2 z, float2 t) {
    const float2 r = rcp_pair(add2(t, C.one));
    const float2 q = mul2(t, r);
    return make_float2(z.x >= 0.f ? r.x : q.x, z.y >= 0.f ? r.y : q.y);
}

}  // namespace gdn
