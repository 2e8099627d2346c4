// gdn_linrec.cuh -- the gated linear recurrence's per-element arithmetic, shared by the prompt,
// single token and gradient kernels so that they agree bit for bit.  Two channels at a time, in
// packed operations.
//
//     r = sigmoid(a_gate), w = K r, K = decay softplus(a_param):  a = e^-w, m = 1 - a   (or a = r, m = 1 - r)
//     s = sqrt((1 - a)(1 + a)) | m | 1,   b = s x sigmoid(x_gate),   h <- a h + b,   y = h act(z)
#pragma once

#include <float.h>
#include <limits.h>

#include "../../include/gdn_linrec.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace linrec {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg(const float2& v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 sub(const float2& a, const float2& b) { return __fadd2_rn(a, neg(b)); }

__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// K of a channel.  Past fp32's range the largest finite value stands for it: a gate that is not 0
// still forgets at once, but a gate of 0 keeps the state and is not 0 times infinity.
__device__ __forceinline__ float rate_of(float a_param, float decay) {
    const float k = __fmul_rn(decay, __fadd_rn(fmaxf(a_param, 0.f), log1pf(expf(-fabsf(a_param)))));
    return k > FLT_MAX ? FLT_MAX : k;
}

// sigmoid(g) and, where asked for, 1 - sigmoid(g) = e^-g sigmoid(g) with its own relative accuracy.
__device__ __forceinline__ float2 sigmoid2(const float2& g, float2& e) {
    const float2 v = __fmul2_rn(g, both(-kLog2e));
    e = make_float2(ex2(v.x), ex2(v.y));
    const float2 d = __fadd2_rn(e, both(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
__device__ __forceinline__ float2 sigmoid2(const float2& g) {
    float2 e;
    return sigmoid2(g, e);
}
// The product is 0 times infinity for far negative g, where 1 stands for it.
__device__ __forceinline__ float2 rest2(const float2& e, const float2& q) {
    const float2 m = __fmul2_rn(e, q);
    constexpr float far = 1.2676506002282294e30f;  // 2^100
    return make_float2(e.x > far ? 1.f : m.x, e.y > far ? 1.f : m.y);
}

// m = 1 - e^-w and a = e^-w for w >= 0.  Below 1/2: m = w + w^2 q(w), q the interpolation of
// ((1 - e^-w) / w - 1) / w of degree 4 (Chebyshev nodes on [0, 1/2] for the series of degree 5; 3e-9 of m), and a = 1 - m,
// rounded once.  Above: a by the hardware exponential and m = 1 - a.
constexpr float kNear = 0.5f;
__device__ __forceinline__ float2 near2(const float2& w) {
    float2 q = __ffma2_rn(both(-0.0011234042467549443f), w, both(0.008189613930881023f));
    q = __ffma2_rn(q, w, both(-0.04163007438182831f));
    q = __ffma2_rn(q, w, both(0.16666242480278015f));
    q = __ffma2_rn(q, w, both(-0.4999998211860657f));
    return __ffma2_rn(__fmul2_rn(w, w), q, w);
}
__device__ __forceinline__ void far1(float w, float& a, float& m) {
    const float e = ex2(__fmul_rn(w, -kLog2e));
    if (!(w < kNear)) a = e, m = __fadd_rn(1.f, -e);
}
__device__ __forceinline__ void decay2(const float2& w, float2& a, float2& m) {
    m = near2(w);
    a = __fadd2_rn(both(1.f), neg(m));
    if (!(fmaxf(w.x, w.y) < kNear)) far1(w.x, a.x, m.x), far1(w.y, a.y, m.y);
}

// 1 - a^2
__device__ __forceinline__ float2 rest_of_square(const float2& a, const float2& m) { return __ffma2_rn(m, a, m); }

// b = s v of one token.
__device__ __forceinline__ float2 intake2(int scale, const float2& a, const float2& m, const float2& v) {
    if (scale == GDN_SCALE_ONE) return v;
    if (scale == GDN_SCALE_LINEAR) return __fmul2_rn(m, v);
    const float2 t = rest_of_square(a, m);
    return __fmul2_rn(make_float2(sqrt_approx(t.x), sqrt_approx(t.y)), v);
}

// The argument of the sigmoid in act(z).
constexpr float kGelu1 = 1.5957691216057308f, kGelu3 = 0.07135481282553144f;  // 2 sqrt(2 / pi), times 0.044715
__device__ __forceinline__ float2 inner2(int act, const float2& z) {
    return act == GDN_ACT_GELU ? __fmul2_rn(z, __ffma2_rn(__fmul2_rn(z, z), both(kGelu3), both(kGelu1))) : z;
}
__device__ __forceinline__ float2 act2(int act, const float2& z) { return __fmul2_rn(z, sigmoid2(inner2(act, z))); }
// act(z) and its slope p + z p (1 - p) inner'(z).
__device__ __forceinline__ float2 act2(int act, const float2& z, float2& slope) {
    float2 e;
    const float2 p = sigmoid2(inner2(act, z), e), r = rest2(e, p), f = __fmul2_rn(z, p);
    float2 g = __fmul2_rn(f, r);
    if (act == GDN_ACT_GELU) g = __fmul2_rn(g, __ffma2_rn(__fmul2_rn(z, z), both(3.f * kGelu3), both(kGelu1)));
    // r is 0 far enough out; where z^2 is past fp32 its product is not
    slope = make_float2(r.x == 0.f || p.x == 0.f ? p.x : __fadd_rn(p.x, g.x), r.y == 0.f || p.y == 0.f ? p.y : __fadd_rn(p.y, g.y));
    return f;
}

struct Params {
    int N, T, C;
    int scale, act;
    float decay;
    const void *x, *ag, *xg, *z;
    int64_t ldx, lda, ldg, ldz;
    const float* ap;
    const int32_t* cu;
    float* state;
    const int32_t* idx;
    int num_slots;
    const int32_t* has_init;
    void* y;
};

__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// a and b of one token's pair of channels.
__device__ __forceinline__ void step2(const Params& p, const float2& K, const float2& ag, const float2& xg, const float2& x,
                                      float2& a, float2& b) {
    float2 e, m;
    const float2 r = sigmoid2(ag, e);
    if (p.ap) decay2(__fmul2_rn(K, r), a, m);
    else a = r, m = rest2(e, r);
    b = intake2(p.scale, a, m, p.xg ? __fmul2_rn(x, sigmoid2(xg)) : x);
}

// Bounds of sequence n, whatever cu_seqlens holds.
__device__ __forceinline__ void bounds(const int32_t* cu, int n, int T, int& bos, int& eos) {
    bos = max(0, min(__ldg(cu + n), T));
    eos = max(bos, min(__ldg(cu + n + 1), T));
}

}  // namespace linrec
}  // namespace gdn
