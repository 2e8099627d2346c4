// gdn_conv_bwd.cu -- gradient of the short causal depthwise conv.
//
//     pre_t = bias + sum_i w_i x_{t-W+1+i},   p_t = d_y_t act'(pre_t)
//     dx_r  = sum_i w_i p_{r+W-1-i},  dw_i = sum_t p_t x_{t-W+1+i},  dbias = sum_t p_t
//
// (p is 0 behind its sequence's end; the W-1 rows before the sequence are its initial state and
// get d_init_state by the same sum; the last W-1 rows of (initial state ++ sequence) get
// d_final_state on top.)  x and d_y are read once and dx is written once: HBM bounds it.
//
// A thread owns 4 channels (two packed pairs) and walks a range of tokens forwards with the last
// W-1 rows of x and of p in registers: row t - (W-1) of dx is complete when p_t is known.  A
// range is T / K tokens whatever sequences it crosses, so ragged batches balance; it re-reads
// W-1 rows on either side.  x and d_y pass through a ring of asynchronous copies in shared memory,
// thread-private (no barriers), two blocks of 8 (fp32: 4) tokens: taps, window and sums leave no registers
// to hold loads in flight.  The dw and dbias sums stay in registers until the end: one row of partials
// per range, which the second kernel adds up in order.
#include <limits.h>

#include "../../include/gdn_layer.h"
#include "gdn_async.cuh"
#include "gdn_host.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

struct ConvBwdParams {
    int N, T, C, K, act;
    const void *x, *h0, *dy, *dhT;
    const float *w, *bias;
    const int32_t* cu;
    void *dx, *dh0;
    float* part;  // [K, W + 1, C]
    float *dw, *db;
};

// Four channels as two packed pairs.
struct Quad {
    float2 a, b;
};
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    using type = uint2;
};
template <>
struct Raw<float> {
    using type = uint4;
};
__device__ __forceinline__ Quad quad(const uint2& u) {
    return {make_float2(bf_lo(u.x), bf_hi(u.x)), make_float2(bf_lo(u.y), bf_hi(u.y))};
}
__device__ __forceinline__ Quad quad(const uint4& u) {
    return {make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), make_float2(__uint_as_float(u.z), __uint_as_float(u.w))};
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const Quad& q) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(bf_pack(q.a.x, q.a.y), bf_pack(q.b.x, q.b.y)));
}
__device__ __forceinline__ void store(float* p, const Quad& q) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(q.a.x, q.a.y, q.b.x, q.b.y));
}
__device__ __forceinline__ void copy_async(uint2* to, const void* from) { copy8_async(to, from); }
__device__ __forceinline__ void copy_async(uint4* to, const void* from) { copy16_async(to, from); }
__device__ __forceinline__ Quad zero() { return {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}; }
__device__ __forceinline__ Quad fma(const Quad& u, const Quad& v, const Quad& w) {
    return {__ffma2_rn(u.a, v.a, w.a), __ffma2_rn(u.b, v.b, w.b)};
}
__device__ __forceinline__ Quad mul(const Quad& u, const Quad& v) { return {__fmul2_rn(u.a, v.a), __fmul2_rn(u.b, v.b)}; }
__device__ __forceinline__ Quad add(const Quad& u, const Quad& v) { return {__fadd2_rn(u.a, v.a), __fadd2_rn(u.b, v.b)}; }

// silu'(x) = s (1 + x (1 - s)), s = sigmoid(x)
__device__ __forceinline__ float2 dsilu(const float2& x) {
    const float2 one = make_float2(1.f, 1.f), e = __fmul2_rn(x, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), one);
    const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    return __fmul2_rn(s, __ffma2_rn(x, __ffma2_rn(s, make_float2(-1.f, -1.f), one), one));
}

template <typename T, int W>
__global__ void __launch_bounds__(128, W <= 4 ? 4 : 2) conv_bwd_kernel(const __grid_constant__ ConvBwdParams p) {
    using R = typename Raw<T>::type;
    constexpr int WM = W - 1, U = sizeof(R) == 8 ? 8 : 4, NS = 2;  // ring: NS blocks of U tokens, 32 KB
    __shared__ R ring[NS][U][2][128];
    const int c0 = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
    if (c0 >= p.C) return;
    const int k = blockIdx.y;
    const int lo = (int)((int64_t)p.T * k / p.K), hi = (int)((int64_t)p.T * (k + 1) / p.K);
    const bool tail = k == p.K - 1;
    const T* x = static_cast<const T*>(p.x) + c0;
    const T* dy = static_cast<const T*>(p.dy) + c0;
    T* dx = static_cast<T*>(p.dx) + c0;
    auto rd = [&](const T* b, int64_t row) { return __ldcs(reinterpret_cast<const R*>(b + row * p.C)); };
    Quad w[W], bias = zero();
    {
        float f[4 * W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p.w + (int64_t)c0 * W) + i);
            f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = {make_float2(f[i], f[W + i]), make_float2(f[2 * W + i], f[3 * W + i])};
        if (p.bias)
            bias = {make_float2(__ldg(p.bias + c0), __ldg(p.bias + c0 + 1)),
                    make_float2(__ldg(p.bias + c0 + 2), __ldg(p.bias + c0 + 3))};
    }
    Quad dw[W], db = zero();
#pragma unroll
    for (int i = 0; i < W; ++i) dw[i] = zero();

    // the first sequence that may have tokens (or, empty, its place) at or behind lo
    int n = 0;
    for (int b = p.N; n < b;) {
        const int mid = (n + b) >> 1;
        if (__ldg(p.cu + mid + 1) >= lo) b = mid; else n = mid + 1;
    }
    for (; n < p.N; ++n) {
        const int bos = max(0, min(__ldg(p.cu + n), p.T)), eos = max(bos, min(__ldg(p.cu + n + 1), p.T));
        if (bos >= hi && !tail) break;
        T* dh = p.dh0 ? static_cast<T*>(p.dh0) + (int64_t)n * WM * p.C + c0 : nullptr;
        const T* dt = p.dhT ? static_cast<const T*>(p.dhT) + (int64_t)n * WM * p.C + c0 : nullptr;
        const T* h0 = p.h0 ? static_cast<const T*>(p.h0) + (int64_t)n * WM * p.C + c0 : nullptr;
        if (bos == eos) {
            if (bos >= lo && dh)
                for (int i = 0; i < WM; ++i) store(dh + (int64_t)i * p.C, dt ? quad(rd(dt, i)) : zero());
            continue;
        }
        const int s = max(bos, lo), e = min(eos, hi);
        if (s >= e) continue;
        Quad win[WM], pw[WM];  // x at t-W+1 .. t-1, p at t-1 .. t-W+1
#pragma unroll
        for (int i = 0; i < WM; ++i) {
            const int r = s - WM + i;
            win[i] = r >= bos ? quad(rd(x, r)) : h0 ? quad(rd(h0, r - bos + WM)) : zero();
            pw[i] = zero();
        }
        // one token: p from x and d_y, the weights' sums, then row t - (W-1) of dx
        auto point = [&](const Quad& xc, const Quad& dyc, bool own) -> Quad {
            Quad pt = dyc;
            if (p.act) {
                Quad pre = bias;
#pragma unroll
                for (int i = 0; i < WM; ++i) pre = fma(w[i], win[i], pre);
                pre = fma(w[WM], xc, pre);
                pt = mul(dyc, {dsilu(pre.a), dsilu(pre.b)});
            }
            if (own) {
#pragma unroll
                for (int i = 0; i < WM; ++i) dw[i] = fma(pt, win[i], dw[i]);
                dw[WM] = fma(pt, xc, dw[WM]);
                db = add(db, pt);
            }
            return pt;
        };
        auto row = [&](const Quad& pt) {
            Quad acc = mul(w[0], pt);
#pragma unroll
            for (int i = 1; i < W; ++i) acc = fma(w[i], pw[i - 1], acc);
            return acc;
        };
        auto slide = [&](const Quad& xc, const Quad& pt) {
#pragma unroll
            for (int i = 0; i + 1 < WM; ++i) win[i] = win[i + 1];
            win[WM - 1] = xc;
#pragma unroll
            for (int i = WM - 1; i > 0; --i) pw[i] = pw[i - 1];
            pw[0] = pt;
        };
        // the ring's tokens: the segment's own and, for the last rows of dx, the W - 1 behind it
        const int loaded = min(e + WM, eos) - s, steps = e + WM - s;
        auto copy = [&](int i) {
            const T* xs = x + (int64_t)(s + i * U) * p.C;
            const T* ys = dy + (int64_t)(s + i * U) * p.C;
            const int64_t C = p.C;
            if ((i + 1) * U <= loaded) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    copy_async(&ring[i % NS][u][0][threadIdx.x], xs + u * C);
                    copy_async(&ring[i % NS][u][1][threadIdx.x], ys + u * C);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i * U + u < loaded) {
                        copy_async(&ring[i % NS][u][0][threadIdx.x], xs + u * C);
                        copy_async(&ring[i % NS][u][1][threadIdx.x], ys + u * C);
                    }
            }
            copy_commit();
        };
        auto any = [&](int t, const R& xr, const R& yr) {  // a token near the segment's ends
            Quad xc = zero(), pt = zero();
            if (t < eos) {
                xc = quad(xr);
                pt = point(xc, quad(yr), t < e);
            }
            const int r = t - WM;
            if (r >= s || s == bos) {
                Quad acc = row(pt);
                const int jf = r - eos + WM;
                if (dt && jf >= 0) acc = add(acc, quad(rd(dt, jf)));
                if (r >= s) store(dx + (int64_t)r * p.C, acc);
                else if (dh) store(dh + (int64_t)(r - bos + WM) * p.C, acc);
            }
            slide(xc, pt);
        };
#pragma unroll
        for (int i = 0; i < NS - 1; ++i) copy(i);
        for (int i = 0; i * U < steps; ++i) {
            copy(i + NS - 1);
            copy_wait<NS - 1>();
            const int t = s + i * U;
            if (t >= s + WM && t + U <= e) {  // all the segment's own, all with a row of dx (d_final_state meets rows complete at t >= eos)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Quad xc = quad(ring[i % NS][u][0][threadIdx.x]), pt = point(xc, quad(ring[i % NS][u][1][threadIdx.x]), true);
                    store(dx + (int64_t)(t + u - WM) * p.C, row(pt));
                    slide(xc, pt);
                }
            } else {
#pragma unroll 1
                for (int u = 0; u < U; ++u)
                    if (t + u < e + WM) any(t + u, ring[i % NS][u][0][threadIdx.x], ring[i % NS][u][1][threadIdx.x]);
            }
        }
        copy_wait<0>();
    }
    float* out = p.part + (int64_t)k * (W + 1) * p.C + c0;
#pragma unroll
    for (int i = 0; i < W; ++i) store(out + (int64_t)i * p.C, dw[i]);
    store(out + (int64_t)W * p.C, db);
}

// dweight [C, W] and dbias [C]: the ranges' partials.  A CTA takes 16 float4 columns of one tap;
// thread (slice, column) adds ranges slice, slice + 16, .., then a thread per column the slices in order.
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(int W, int C, int K, const float* __restrict__ part,
                                                           float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float4 sums[16][16];
    const int x = threadIdx.x & 15, slice = threadIdx.x >> 4, i = blockIdx.y;
    const int c = (blockIdx.x * 16 + x) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v) { s.x = __fadd_rn(s.x, v.x), s.y = __fadd_rn(s.y, v.y), s.z = __fadd_rn(s.z, v.z), s.w = __fadd_rn(s.w, v.w); };
    if (c < C) {
#pragma unroll 4
        for (int k = slice; k < K; k += 16) add(*reinterpret_cast<const float4*>(part + ((int64_t)k * (W + 1) + i) * C + c));
    }
    sums[slice][x] = s;
    __syncthreads();
    if (slice || c >= C) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) add(sums[k][x]);
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (i < W) dw[(int64_t)(c + e) * W + i] = v[e];
        else if (db) db[c + e] = v[e];
    }
}

// Token ranges: one wave of CTAs of 128 x 4 channels, four an SM, but no range under 16 tokens.
int conv_ranges(int T, int C) {
    const int cols = (C + 511) / 512;
    const int most = (T + 15) / 16;
    const int want = kSMs * 4 / cols > 1 ? kSMs * 4 / cols : 1;
    return want < most ? want : (most > 1 ? most : 1);
}

gdn_status check_conv_bwd(const gdn_conv_shape* s) {
    if (!s) return GDN_ERR_INVALID_ARG;
    if (s->N < 0 || s->T_total < 0 || s->C <= 0) return GDN_ERR_INVALID_ARG;
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (s->W < 2 || s->W > 8) return GDN_ERR_UNSUPPORTED;
    if (s->C % (s->dtype == GDN_BF16 ? 8 : 4)) return GDN_ERR_UNSUPPORTED;
    if (s->T_total > INT_MAX - 64 || (long long)s->T_total * s->C >= (1LL << 40)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

template <typename T>
gdn_status conv_bwd_launch(int W, dim3 grid, cudaStream_t s, const ConvBwdParams& p) {
    switch (W) {
        case 2: conv_bwd_kernel<T, 2><<<grid, 128, 0, s>>>(p); break;
        case 3: conv_bwd_kernel<T, 3><<<grid, 128, 0, s>>>(p); break;
        case 4: conv_bwd_kernel<T, 4><<<grid, 128, 0, s>>>(p); break;
        case 5: conv_bwd_kernel<T, 5><<<grid, 128, 0, s>>>(p); break;
        case 6: conv_bwd_kernel<T, 6><<<grid, 128, 0, s>>>(p); break;
        case 7: conv_bwd_kernel<T, 7><<<grid, 128, 0, s>>>(p); break;
        case 8: conv_bwd_kernel<T, 8><<<grid, 128, 0, s>>>(p); break;
        default: return GDN_ERR_UNSUPPORTED;
    }
    return launch_status();
}

}  // namespace
}  // namespace gdn

extern "C" size_t gdn_causal_conv1d_bwd_workspace_size(const gdn_conv_shape* shape) {
    using namespace gdn;
    if (check_conv_bwd(shape) != GDN_OK) return 0;
    return (size_t)conv_ranges(shape->T_total, shape->C) * (shape->W + 1) * shape->C * sizeof(float);
}

extern "C" gdn_status gdn_causal_conv1d_bwd(const gdn_conv_shape* shape, const void* x, const float* weight,
                                            const float* bias, const int32_t* cu_seqlens, const void* init_state,
                                            const void* d_y, const void* d_final_state, void* dx, float* dweight,
                                            float* dbias, void* d_init_state, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    using namespace gdn;
    gdn_status st = check_conv_bwd(shape);
    if (st != GDN_OK) return st;
    const bool rows = shape->T_total > 0;
    if (rows && shape->N == 0) return GDN_ERR_INVALID_ARG;
    if (!weight || !cu_seqlens || !dweight || (rows && (!x || !d_y || !dx))) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(d_y) || !aligned16(dx) || !aligned16(init_state) || !aligned16(d_final_state) ||
        !aligned16(d_init_state) || !aligned16(weight) || !aligned4(bias) || !aligned4(cu_seqlens) ||
        !aligned4(dweight) || !aligned4(dbias))
        return GDN_ERR_INVALID_ARG;
    if (dx && (dx == x || dx == d_y)) return GDN_ERR_INVALID_ARG;
    if (d_init_state && (d_init_state == init_state || d_init_state == d_final_state)) return GDN_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < gdn_causal_conv1d_bwd_workspace_size(shape))
        return GDN_ERR_WORKSPACE;
    const int W = shape->W, C = shape->C;
    ConvBwdParams p{shape->N, shape->T_total, C, conv_ranges(shape->T_total, C), shape->activation,
                    x, init_state, d_y, d_final_state, weight, bias, cu_seqlens, dx, d_init_state,
                    static_cast<float*>(workspace), dweight, dbias};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)((C + 511) / 512), (unsigned)p.K);
    st = shape->dtype == GDN_BF16 ? conv_bwd_launch<__nv_bfloat16>(W, grid, s, p) : conv_bwd_launch<float>(W, grid, s, p);
    if (st != GDN_OK) return st;
    conv_bwd_sum_kernel<<<dim3((unsigned)((C + 63) / 64), (unsigned)(W + 1)), 256, 0, s>>>(W, C, p.K, p.part, dweight, dbias);
    return launch_status();
}
