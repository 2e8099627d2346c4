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

// K of a channel.  Near and past fp32's range kMost stands for it: a gate that is not 0 still forgets at once, but a gate of 0 keeps
// the state and is not 0 times infinity, and K r stays finite where r rounds past 1 (the gradient's e^-w w is not 0 times infinity).
constexpr float kMost = 3e38f;
__device__ __forceinline__ float rate_of(float a_param, float decay) {
    const float k = __fmul_rn(decay, __fadd_rn(fmaxf(a_param, 0.f), log1pf(expf(-fabsf(a_param)))));
    return k > kMost ? kMost : k;
}

// The largest of three, or NaN if one is.
__device__ __forceinline__ float most_or_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 1 / (1 + 2^v), and 2^v.
__device__ __forceinline__ float2 logistic2(const float2& v, float2& e) {
    e = make_float2(ex2(v.x), ex2(v.y));
    const float2 d = __fadd2_rn(e, both(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
// 1 / (1 + e) and e / (1 + e) for any e, infinity too.
constexpr float kFar = 1.152921504606847e18f;  // 2^60
__device__ __forceinline__ void apart(float e, float& r, float& r1) {
    r = rcp_approx(__fadd_rn(1.f, e));
    r1 = e > 1e36f ? 1.f : __fmul_rn(e, r);
}

// sigmoid(g) = r and sigmoid(i) = p with one reciprocal for both, 1 / ((1 + 2^v) (1 + 2^u)): the special function unit, which
// takes two cycles a warp for a reciprocal or a root and one for an exponential, bounds the prompts' kernel next to HBM.
// r1, p1: 1 - r and 1 - p.  Where a power is past 2^60 and their product might leave fp32's range, or one is not a number and would
// make the other gate's sigmoid so too, each has its own.
template <int NP>
__device__ __forceinline__ void two_sigmoids(const float2 (&g)[NP], const float2 (&i)[NP], float2 (&r)[NP], float2 (&p)[NP], float2 (&r1)[NP], float2 (&p1)[NP]) {
    float2 e[NP], f[NP];
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const float2 v = __fmul2_rn(g[k], both(-kLog2e)), u = __fmul2_rn(i[k], both(-kLog2e));
        most = most_or_nan(most_or_nan(most, v.x, v.y), u.x, u.y);
        e[k] = make_float2(ex2(v.x), ex2(v.y)), f[k] = make_float2(ex2(u.x), ex2(u.y));
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const float2 d = __fadd2_rn(e[k], both(1.f)), c = __fadd2_rn(f[k], both(1.f)), D = __fmul2_rn(d, c);
        const float2 R = make_float2(rcp_approx(D.x), rcp_approx(D.y));
        r[k] = __fmul2_rn(R, c), p[k] = __fmul2_rn(R, d);
        r1[k] = __fmul2_rn(e[k], r[k]), p1[k] = __fmul2_rn(f[k], p[k]);
    }
    if (!(most <= 60.f)) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (!(most_or_nan(0.f, e[k].x, f[k].x) <= kFar)) apart(e[k].x, r[k].x, r1[k].x), apart(f[k].x, p[k].x, p1[k].x);
            if (!(most_or_nan(0.f, e[k].y, f[k].y) <= kFar)) apart(e[k].y, r[k].y, r1[k].y), apart(f[k].y, p[k].y, p1[k].y);
        }
    }
}
// sigmoid(g) = r alone, and 1 - r.
template <int NP>
__device__ __forceinline__ void one_sigmoid(const float2 (&g)[NP], float2 (&r)[NP], float2 (&r1)[NP]) {
    float2 e[NP];
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const float2 v = __fmul2_rn(g[k], both(-kLog2e));
        most = fmaxf(most, fmaxf(v.x, v.y));
        r[k] = logistic2(v, e[k]), r1[k] = __fmul2_rn(e[k], r[k]);
    }
    if (most > 60.f) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (e[k].x > kFar) apart(e[k].x, r[k].x, r1[k].x);
            if (e[k].y > kFar) apart(e[k].y, r[k].y, r1[k].y);
        }
    }
}

// The decay without an a_param, sigmoid(g).  Next to 1 it is 1 minus its rest r1, rounded once, and so never past 1: r, from the reciprocal that two
// gates share, is up to an ulp off 1 on either side, which a kept state would take at every token (4096 open gates: 5e-4 of it).  Costs
// 16 prompts, 32768 x 4096, bf16, 231 -> 239 us with an x_gate and 193 -> 195 without, the gradient 693 -> 713 and 541 -> 549.
template <int NP>
__device__ __forceinline__ void forget(const float2 (&r)[NP], const float2 (&r1)[NP], float2 (&a)[NP]) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const float2 o = __ffma2_rn(r1[k], both(-1.f), both(1.f));
        a[k] = make_float2(r1[k].x < 0.5f ? o.x : r[k].x, r1[k].y < 0.5f ? o.y : r[k].y);
    }
}

// m = 1 - e^-w and a = e^-w for w >= 0.  Below 1/4: m = w + w^2 q(w), q the interpolation of (1 - e^-w - w) / w^2 of
// degree 3 at Chebyshev's nodes on [0, 1/4] (1.2e-8 of m), and a = 1 - m, rounded once.  Above: a by the
// hardware exponential and m = 1 - a.  w = K r, and r, an approximation, is past 1 by 2^-22 at most: channels whose K is below 1/4
// by 2^-20 of it have no far tokens.
constexpr float kNear = 0.25f;
__device__ __forceinline__ float2 near2(const float2& w) {
    float2 q = __ffma2_rn(both(0.00767176877707243f), w, both(-0.041564859449863434f));
    q = __ffma2_rn(q, w, both(0.1666616052389145f));
    q = __ffma2_rn(q, w, both(-0.4999999701976776f));
    return __ffma2_rn(__fmul2_rn(w, w), q, w);
}
__device__ __forceinline__ void far1(float w, float& a, float& m) {
    const float e = ex2(__fmul_rn(w, -kLog2e));
    if (!(w < kNear)) a = e, m = __fadd_rn(1.f, -e);
}
template <int NP>
__device__ __forceinline__ void decays(bool far, const float2 (&w)[NP], float2 (&a)[NP], float2 (&m)[NP]) {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        m[e] = near2(w[e]);
        a[e] = __ffma2_rn(m[e], both(-1.f), both(1.f));
    }
    if (!far) return;
#pragma unroll
    for (int e = 0; e < NP; ++e) far1(w[e].x, a[e].x, m[e].x), far1(w[e].y, a[e].y, m[e].y);
}

// 1 - a^2
__device__ __forceinline__ float2 rest_of_square(const float2& a, const float2& m) { return __ffma2_rn(m, a, m); }

// act(z) = z sigmoid(i(z)); inner2 gives -i(z) log2(e), the exponent that the sigmoid takes.
constexpr float kGelu1 = 1.5957691216057308f, kGelu3 = 0.07135481282553144f;  // i = z (2 sqrt(2 / pi) + 0.044715 times that z^2)
__device__ __forceinline__ float2 inner2(int act, const float2& z) {
    if (act != GDN_ACT_GELU) return __fmul2_rn(z, both(-kLog2e));
    return __fmul2_rn(z, __ffma2_rn(__fmul2_rn(z, z), both(-kLog2e * kGelu3), both(-kLog2e * kGelu1)));
}
// f = act(z) and its slope p + z p (1 - p) i'(z), where p and 1 - p have their own relative accuracy; far out, where
// these products leave fp32's range, the slope is 0 or 1.
template <int NP>
__device__ __forceinline__ void act_slope(int act, const float2 (&z)[NP], float2 (&f)[NP], float2 (&slope)[NP]) {
    float2 v[NP];
    float most = 0.f;
    if (act == GDN_ACT_GELU) {
#pragma unroll
        for (int k = 0; k < NP; ++k) v[k] = inner2(GDN_ACT_GELU, z[k]), slope[k] = __ffma2_rn(__fmul2_rn(z[k], z[k]), both(3.f * kGelu3), both(kGelu1));
    } else {
#pragma unroll
        for (int k = 0; k < NP; ++k) v[k] = inner2(GDN_ACT_SILU, z[k]), slope[k] = both(1.f);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        most = fmaxf(most, fmaxf(fabsf(v[k].x), fabsf(v[k].y)));
        float2 e;
        const float2 p = logistic2(v[k], e);
        f[k] = __fmul2_rn(z[k], p);
        slope[k] = __ffma2_rn(__fmul2_rn(f[k], __fmul2_rn(e, p)), slope[k], p);
    }
    if (most > 120.f) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (fabsf(v[k].x) > 120.f) slope[k].x = v[k].x > 0.f ? 0.f : 1.f;
            if (fabsf(v[k].y) > 120.f) slope[k].y = v[k].y > 0.f ? 0.f : 1.f;
        }
    }
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
    int ranked;                  // prompts: take the sequences in order of length
    int64_t sx, sa, sg, sz, sy;  // prompts: bytes from a tile's row of x, a_gate, x_gate, z, y to the next tile's
};

// Which of a call's options a kernel knows at compile time.  With all of them as branches the values that meet
// behind each branch are moved about (16 prompts, 32768 x 4096, when it was chosen: 307 us, so 283); all combinations would be 36 kernels of
// each.  kBothGates: a_param, x_gate, scale sqrt; kForget: neither, scale linear; kAny: asks at run time.  The bits are the same.
enum Kind { kAny, kBothGates, kForget };
template <Kind KIND>
__device__ __forceinline__ bool has_param(const Params& p) { return KIND == kAny ? p.ap != nullptr : KIND == kBothGates; }
template <Kind KIND>
__device__ __forceinline__ bool has_gate(const Params& p) { return KIND == kAny ? p.xg != nullptr : KIND == kBothGates; }
template <Kind KIND>
__device__ __forceinline__ int scale_of(const Params& p) { return KIND == kAny ? p.scale : KIND == kBothGates ? GDN_SCALE_SQRT : GDN_SCALE_LINEAR; }
inline Kind kind_of(const Params& p) {
    if (p.ap && p.xg && p.scale == GDN_SCALE_SQRT) return kBothGates;
    return !p.ap && !p.xg && p.scale == GDN_SCALE_LINEAR ? kForget : kAny;
}

// Whether a channel of these rates has far tokens.
template <int NP>
__device__ __forceinline__ bool any_far(const float2 (&K)[NP]) {
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < NP; ++e) most = fmaxf(most, fmaxf(K[e].x, K[e].y));
    return most >= kNear * (1.f - 0x1p-20f);
}

// a and b of NP pairs (neighbouring channels, or one channel's tokens).  Options are branches around whole loops, so that
// the pairs' operations overlap.
template <Kind KIND, int NP>
__device__ __forceinline__ void steps(const Params& p, bool far, const float2 (&K)[NP], const float2 (&ag)[NP], const float2 (&xg)[NP],
                                      const float2 (&x)[NP], float2 (&a)[NP], float2 (&b)[NP]) {
    float2 m[NP], r[NP], r1[NP];
    if (has_gate<KIND>(p)) {
        float2 p1[NP];
        two_sigmoids(ag, xg, r, b, r1, p1);
#pragma unroll
        for (int e = 0; e < NP; ++e) b[e] = __fmul2_rn(x[e], b[e]);
    } else {
        one_sigmoid(ag, r, r1);
#pragma unroll
        for (int e = 0; e < NP; ++e) b[e] = x[e];
    }
    if (has_param<KIND>(p)) {
        float2 w[NP];
#pragma unroll
        for (int e = 0; e < NP; ++e) w[e] = __fmul2_rn(K[e], r[e]);
        decays(far, w, a, m);
    } else {
        forget(r, r1, a);
#pragma unroll
        for (int e = 0; e < NP; ++e) m[e] = r1[e];
    }
    if (scale_of<KIND>(p) == GDN_SCALE_SQRT) {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const float2 t = rest_of_square(a[e], m[e]);
            b[e] = __fmul2_rn(make_float2(sqrt_approx(t.x), sqrt_approx(t.y)), b[e]);
        }
    } else if (scale_of<KIND>(p) == GDN_SCALE_LINEAR) {
#pragma unroll
        for (int e = 0; e < NP; ++e) b[e] = __fmul2_rn(m[e], b[e]);
    }
}
// y = h act(z) of NP pairs.
template <int NP>
__device__ __forceinline__ void branch(int act, const float2 (&z)[NP], float2 (&h)[NP]) {
    float2 e;
    if (act == GDN_ACT_GELU) {
#pragma unroll
        for (int k = 0; k < NP; ++k) h[k] = __fmul2_rn(h[k], __fmul2_rn(z[k], logistic2(inner2(GDN_ACT_GELU, z[k]), e)));
    } else {
#pragma unroll
        for (int k = 0; k < NP; ++k) h[k] = __fmul2_rn(h[k], __fmul2_rn(z[k], logistic2(inner2(GDN_ACT_SILU, z[k]), e)));
    }
}

// Bounds of sequence n, whatever cu_seqlens holds.
__device__ __forceinline__ void bounds(const int32_t* cu, int n, int T, int& bos, int& eos) {
    bos = max(0, min(__ldg(cu + n), T));
    eos = max(bos, min(__ldg(cu + n + 1), T));
}

}  // namespace linrec
}  // namespace gdn
