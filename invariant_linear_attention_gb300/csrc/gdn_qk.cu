// gdn_qk.cu -- norm of the heads of q and k and rotation by position, and its gradient.
//
//     n = x r w,  r = (c sum x^2 + eps)^-1/2,  c = 1/d or 1;   out = R n
//     g = w R^T d_out:   dx = r g - x r^3 c sum(g x),   dw = sum over rows of x r R^T d_out
//
// (R: the rotation of the pairs.)  Every value is read once and written once: HBM bounds it.
//
// A row (one head of one token) is cut into units of two 16-byte chunks that hold whole pairs:
// chunks (u, u + rotary_dim/2) of the halves form, two neighbouring chunks otherwise.  A lane
// takes one unit, a power-of-two group of lanes one row, so a rotation needs no other lane and
// the sum of squares a fixed butterfly.  A warp takes as many heads of one token as it has
// groups per pass, several passes' loads at once, and goes on to the token's other heads with the same
// angles in registers.  Packed pairs of values: issue slots bound the first version (17 a value).
#include "../../include/gdn_layer.h"
#include "gdn_host.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

struct QkParams {
    int64_t T;
    int HQ, HK, d, rd, inter, max_pos;
    float c, eps;
    int64_t ldq, ldk, lddq, lddk;
    const void *q, *k, *dqo, *dko;
    const float *qw, *kw, *cos, *sin;
    const int32_t* pos;
    void *qo, *ko;   // outputs (gradient: dq, dk)
    float* part;     // gradient: [CTAs, 2, d]
    int lpr;         // lanes per row
    int passes;      // head passes a warp takes per item
    int pq, pk;      // head passes of q and of k
    int64_t items;
};

// Where a lane's unit lies: its two chunks' first values, whether each exists, and whether it is rotated.
struct Unit {
    int e0, e1;
    bool has0, has1, rot;
};
template <int VN>
__device__ __forceinline__ Unit unit_of(int u, int d, int rd, int inter) {
    const int hc = rd / (2 * VN);
    Unit r;
    r.rot = u < hc;
    const int first = r.rot ? (inter ? 2 * u : u) : rd / VN + 2 * (u - hc);
    const int second = r.rot && !inter ? u + hc : first + 1;
    r.e0 = first * VN, r.e1 = second * VN;
    r.has0 = r.e0 < d, r.has1 = r.e1 < d;
    return r;
}

// A unit's values as packed pairs: its first chunk in [0, VN / 2), its second behind it.
template <int VN>
__device__ __forceinline__ void unpack_unit(const uint4& a, const uint4& b, float2 (&v)[VN]) {
    float f[VN], g[VN];
    unpack(a, f);
    unpack(b, g);
#pragma unroll
    for (int e = 0; e < VN / 2; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]), v[VN / 2 + e] = make_float2(g[2 * e], g[2 * e + 1]);
}
template <int VN>
__device__ __forceinline__ uint4 pack_half(const float2* v) {
    float f[VN];
#pragma unroll
    for (int e = 0; e < VN / 2; ++e) f[2 * e] = v[e].x, f[2 * e + 1] = v[e].y;
    return pack(f);
}
__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

// The angles of a unit's VN pairs; back: the negative ones.  A unit that is not rotated is not turned
// by 1 and 0 either: that would spread an infinity to its neighbour.
template <int VN>
struct Angles {
    float2 c[VN / 2], s[VN / 2], ns[VN / 2];
    __device__ __forceinline__ void load(const QkParams& p, int64_t row, int u, bool rot, bool back) {
        const float* pc = p.cos + row * (p.rd / 2) + u * VN;
        const float* ps = p.sin + row * (p.rd / 2) + u * VN;
#pragma unroll
        for (int e = 0; e < VN / 2; e += 2) {
            const float4 c4 = rot ? __ldg(reinterpret_cast<const float4*>(pc + 2 * e)) : make_float4(1.f, 1.f, 1.f, 1.f);
            const float4 s4 = rot ? __ldg(reinterpret_cast<const float4*>(ps + 2 * e)) : make_float4(0.f, 0.f, 0.f, 0.f);
            c[e] = make_float2(c4.x, c4.y), c[e + 1] = make_float2(c4.z, c4.w);
            s[e] = make_float2(s4.x, s4.y), s[e + 1] = make_float2(s4.z, s4.w);
        }
#pragma unroll
        for (int e = 0; e < VN / 2; ++e) {
            ns[e] = make_float2(-s[e].x, -s[e].y);
            if (back) {
                const float2 t = s[e];
                s[e] = ns[e], ns[e] = t;
            }
        }
    }
    // (u, v) -> (u c - v s, v c + u s).  Halves: u in the first chunk, v in the second; neighbours: a pair is (u, v).
    template <bool INTER>
    __device__ __forceinline__ void turn(float2 (&v)[VN]) const {
        if constexpr (!INTER) {
#pragma unroll
            for (int e = 0; e < VN / 2; ++e) {
                const float2 a = v[e], b = v[VN / 2 + e];
                v[e] = __ffma2_rn(b, ns[e], __fmul2_rn(a, c[e]));
                v[VN / 2 + e] = __ffma2_rn(a, s[e], __fmul2_rn(b, c[e]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const float2 a = v[e];
                const float ce = e & 1 ? c[e / 2].y : c[e / 2].x, se = e & 1 ? s[e / 2].y : s[e / 2].x, me = e & 1 ? ns[e / 2].y : ns[e / 2].x;
                v[e] = make_float2(__fmaf_rn(a.y, me, __fmul_rn(a.x, ce)), __fmaf_rn(a.x, se, __fmul_rn(a.y, ce)));
            }
        }
    }
};

// A unit's weights (ones where there is no weight).
template <int VN>
__device__ __forceinline__ void load_weight(const float* w, const Unit& un, float2 (&v)[VN]) {
#pragma unroll
    for (int e = 0; e < VN; e += 2) {
        const bool has = w && (e < VN / 2 ? un.has0 : un.has1);
        const float4 t = has ? __ldg(reinterpret_cast<const float4*>(w + (e < VN / 2 ? un.e0 + 2 * e : un.e1 + 2 * e - VN))) : make_float4(1.f, 1.f, 1.f, 1.f);
        v[e] = make_float2(t.x, t.y), v[e + 1] = make_float2(t.z, t.w);
    }
}

__device__ __forceinline__ float group_sum(float s, int lpr) {
    for (int off = 1; off < lpr; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}
template <int VN>
__device__ __forceinline__ float dot(const float2 (&a)[VN], const float2 (&b)[VN]) {
    float2 s = __fmul2_rn(a[0], b[0]);
#pragma unroll
    for (int e = 1; e < VN; ++e) s = __ffma2_rn(a[e], b[e], s);
    return __fadd_rn(s.x, s.y);
}

// The token's angle row, or -1 where it is skipped.
__device__ __forceinline__ int64_t angle_row(const QkParams& p, int64_t t) {
    if (p.rd == 0) return 0;
    const int64_t pos = p.pos ? (int64_t)__ldg(p.pos + t) : t;
    return pos >= 0 && pos < p.max_pos ? pos : -1;
}

// PART: some units are not rotated (whole heads skip the test: 90 us instead of 106 for 32768 x 32 x
// 128).  UR: passes whose loads are in flight together.
template <typename T, bool INTER, bool PART, bool HASW>
__global__ void __launch_bounds__(256) qk_kernel(const __grid_constant__ QkParams p) {
    constexpr int VN = V16<T>::n, UR = 2;
    const int lane = threadIdx.x & 31, u = lane & (p.lpr - 1), sub = lane / p.lpr, hpw = 32 / p.lpr;
    const Unit un = unit_of<VN>(u, p.d, p.rd, p.inter);
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int all = p.pq + p.pk, per = (all + p.passes - 1) / p.passes;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < p.items; it += nwarps) {
        const int64_t t = it / per;
        const int64_t row = angle_row(p, t);
        if (row < 0) continue;
        Angles<VN> an;
        an.load(p, row, u, un.rot, false);
        const int first = (int)(it % per) * p.passes, last = min(first + p.passes, all);
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {  // q, then k
            const int H = side ? p.HK : p.HQ, lo = side ? max(first - p.pq, 0) : first, hi = side ? last - p.pq : min(last, p.pq);
            if (lo >= hi) continue;
            const T* src = (side ? static_cast<const T*>(p.k) + t * p.ldk : static_cast<const T*>(p.q) + t * p.ldq);
            T* dst = (side ? static_cast<T*>(p.ko) : static_cast<T*>(p.qo)) + t * H * p.d;
            float2 w[VN];
            if constexpr (HASW) load_weight<VN>(side ? p.kw : p.qw, un, w);
            for (int ps = lo; ps < hi; ps += UR) {
                uint4 ra[UR], rb[UR];
#pragma unroll
                for (int i = 0; i < UR; ++i) {
                    const int h = (ps + i) * hpw + sub;
                    const bool ok = ps + i < hi && h < H;
                    ra[i] = ok && un.has0 ? ld16_stream(src + h * p.d + un.e0) : none;
                    rb[i] = ok && un.has1 ? ld16_stream(src + h * p.d + un.e1) : none;
                }
#pragma unroll
                for (int i = 0; i < UR; ++i) {
                    if (ps + i >= hi) break;
                    const int h = (ps + i) * hpw + sub;
                    float2 v[VN];
                    unpack_unit<VN>(ra[i], rb[i], v);
                    const float2 r = twice(rsqrtf(__fmaf_rn(group_sum(dot<VN>(v, v), p.lpr), p.c, p.eps)));
#pragma unroll
                    for (int e = 0; e < VN; ++e) {
                        v[e] = __fmul2_rn(v[e], r);
                        if constexpr (HASW) v[e] = __fmul2_rn(v[e], w[e]);
                    }
                    if (!PART || un.rot) an.template turn<INTER>(v);
                    if (h < H && un.has0) st16_stream(dst + h * p.d + un.e0, pack_half<VN>(v));
                    if (h < H && un.has1) st16_stream(dst + h * p.d + un.e1, pack_half<VN>(v + VN / 2));
                }
            }
        }
    }
}

template <typename T, bool INTER, bool PART, bool HASW>
__global__ void __launch_bounds__(256, 2) qk_bwd_kernel(const __grid_constant__ QkParams p) {
    constexpr int VN = V16<T>::n, UR = 2;
    extern __shared__ float acc[];  // [256 / lpr groups][d]
    const int lane = threadIdx.x & 31, u = lane & (p.lpr - 1), sub = lane / p.lpr, hpw = 32 / p.lpr;
    const Unit un = unit_of<VN>(u, p.d, p.rd, p.inter);
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {  // q, then k
        const int H = side ? p.HK : p.HQ, np = side ? p.pk : p.pq;
        const int64_t ld = side ? p.ldk : p.ldq, ldd = side ? p.lddk : p.lddq;
        const T* x = static_cast<const T*>(side ? p.k : p.q);
        const T* dout = static_cast<const T*>(side ? p.dko : p.dqo);
        T* dx = static_cast<T*>(side ? p.ko : p.qo);
        const float* wp = side ? p.kw : p.qw;
        float2 w[VN], sum[VN];
        if constexpr (HASW) {
            load_weight<VN>(wp, un, w);
#pragma unroll
            for (int e = 0; e < VN; ++e) sum[e] = twice(0.f);
        }
        const int per = (np + p.passes - 1) / p.passes;  // items of a token
        for (int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < p.T * per; it += nwarps) {
            const int64_t t = per == 1 ? it : it / per;
            const int first = per == 1 ? 0 : (int)(it % per) * p.passes, last = min(first + p.passes, np);
            const int64_t row = angle_row(p, t);
            if (row < 0) continue;
            Angles<VN> an;
            an.load(p, row, u, un.rot, true);
            const T* src = x + t * ld;
            const T* dsrc = dout + t * H * p.d;
            T* dst = dx + t * ldd;
            for (int ps = first; ps < last; ps += UR) {
                uint4 ra[UR], rb[UR], ga[UR], gb[UR];
#pragma unroll
                for (int i = 0; i < UR; ++i) {
                    const int h = (ps + i) * hpw + sub;
                    const bool ok = ps + i < last && h < H;
                    ra[i] = ok && un.has0 ? ld16_stream(src + h * p.d + un.e0) : none;
                    rb[i] = ok && un.has1 ? ld16_stream(src + h * p.d + un.e1) : none;
                    ga[i] = ok && un.has0 ? ld16_stream(dsrc + h * p.d + un.e0) : none;
                    gb[i] = ok && un.has1 ? ld16_stream(dsrc + h * p.d + un.e1) : none;
                }
#pragma unroll
                for (int i = 0; i < UR; ++i) {
                    if (ps + i >= last) break;
                    const int h = (ps + i) * hpw + sub;
                    float2 v[VN], g[VN];
                    unpack_unit<VN>(ra[i], rb[i], v);
                    unpack_unit<VN>(ga[i], gb[i], g);
                    const float r = rsqrtf(__fmaf_rn(group_sum(dot<VN>(v, v), p.lpr), p.c, p.eps));
                    if (!PART || un.rot) an.template turn<INTER>(g);
                    if constexpr (HASW) {
#pragma unroll
                        for (int e = 0; e < VN; ++e) {
                            sum[e] = __ffma2_rn(__fmul2_rn(v[e], twice(h < H ? r : 0.f)), g[e], sum[e]);
                            g[e] = __fmul2_rn(g[e], w[e]);
                        }
                    }
                    const float gx = group_sum(dot<VN>(g, v), p.lpr);
                    // r (g - x (r sum(g x)) (r c)): with eps = 0 and small rows r^3 is past fp32, these products are not
                    const float f = -__fmul_rn(__fmul_rn(r, gx), __fmul_rn(r, p.c));
#pragma unroll
                    for (int e = 0; e < VN; ++e) v[e] = __fmul2_rn(twice(r), __ffma2_rn(v[e], twice(f), g[e]));
                    if (h < H && un.has0) st16_stream(dst + h * p.d + un.e0, pack_half<VN>(v));
                    if (h < H && un.has1) st16_stream(dst + h * p.d + un.e1, pack_half<VN>(v + VN / 2));
                }
            }
        }
        // the CTA's sum for the weight: its lane groups in ascending order
        if constexpr (HASW) {
            if (!p.part) continue;
            float* mine = acc + (int64_t)(threadIdx.x / p.lpr) * p.d;
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                float* to = mine + (e < VN / 2 ? un.e0 + 2 * e : un.e1 + 2 * e - VN);
                if (e < VN / 2 ? un.has0 : un.has1) to[0] = sum[e].x, to[1] = sum[e].y;
            }
            __syncthreads();
            for (int e = threadIdx.x; e < p.d; e += blockDim.x) {
                float s = 0.f;
                for (int i = 0; i < (int)blockDim.x / p.lpr; ++i) s = __fadd_rn(s, acc[(int64_t)i * p.d + e]);
                p.part[((int64_t)blockIdx.x * 2 + side) * p.d + e] = s;
            }
            __syncthreads();
        }
    }
}

// dweight [d] of q (blockIdx.y 0) and k (1): the CTAs' partials.  A CTA takes 4 float4 columns;
// thread (slice, column) adds partials slice, slice + 64, .., then a thread per column the slices in order.
__global__ void __launch_bounds__(256) qk_bwd_sum_kernel(int d, int ctas, const float* __restrict__ part,
                                                         float* __restrict__ dqw, float* __restrict__ dkw) {
    __shared__ float4 sums[64][4];
    const int x = threadIdx.x & 3, slice = threadIdx.x >> 2, side = blockIdx.y, e = (blockIdx.x * 4 + x) * 4;
    float* out = side ? dkw : dqw;
    if (!out) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v) { s.x = __fadd_rn(s.x, v.x), s.y = __fadd_rn(s.y, v.y), s.z = __fadd_rn(s.z, v.z), s.w = __fadd_rn(s.w, v.w); };
    if (e < d) {
#pragma unroll 4
        for (int i = slice; i < ctas; i += 64) add(*reinterpret_cast<const float4*>(part + ((int64_t)i * 2 + side) * d + e));
    }
    sums[slice][x] = s;
    __syncthreads();
    if (slice || e >= d) return;
    for (int i = 1; i < 64; ++i) add(sums[i][x]);
    out[e] = s.x, out[e + 1] = s.y, out[e + 2] = s.z, out[e + 3] = s.w;
}

gdn_status check_qk(const gdn_qk_shape* s) {
    if (!s) return GDN_ERR_INVALID_ARG;
    if (s->T < 0 || s->HQ <= 0 || s->HK < 0 || s->d <= 0 || s->max_positions < 0) return GDN_ERR_INVALID_ARG;
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    const int vn = s->dtype == GDN_BF16 ? 8 : 4;
    if (s->d % vn || s->d > 256 || s->rotary_dim % (2 * vn)) return GDN_ERR_UNSUPPORTED;
    if (s->norm != GDN_NORM_RMS && s->norm != GDN_NORM_L2) return GDN_ERR_UNSUPPORTED;
    if (s->rotary_dim < 0 || s->rotary_dim > s->d || !(s->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (s->ldq < (int64_t)s->HQ * s->d || s->ldk < (int64_t)s->HK * s->d || s->ldq % vn || s->ldk % vn) return GDN_ERR_INVALID_ARG;
    if (s->T >= (1LL << 31) || (int64_t)(s->HQ + (int64_t)s->HK) >= (1LL << 20)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

QkParams qk_params(const gdn_qk_shape* s) {
    QkParams p{};
    p.T = s->T, p.HQ = s->HQ, p.HK = s->HK, p.d = s->d, p.rd = s->rotary_dim, p.inter = s->interleaved;
    p.max_pos = s->max_positions, p.eps = s->eps, p.ldq = s->ldq, p.ldk = s->ldk;
    p.c = s->norm == GDN_NORM_RMS ? 1.f / (float)s->d : 1.f;
    const int vn = s->dtype == GDN_BF16 ? 8 : 4;
    const int hc = s->rotary_dim / (2 * vn), units = hc + ((s->d - s->rotary_dim) / vn + 1) / 2;
    p.lpr = 1;
    while (p.lpr < units) p.lpr *= 2;
    const int hpw = 32 / p.lpr;
    p.pq = (p.HQ + hpw - 1) / hpw, p.pk = (p.HK + hpw - 1) / hpw;
    return p;
}

gdn_status check_angles(const gdn_qk_shape* s, const float* cos, const float* sin, const int32_t* pos) {
    if (s->rotary_dim == 0) return GDN_OK;
    if (!cos || !sin || !aligned16(cos) || !aligned16(sin) || !aligned4(pos)) return GDN_ERR_INVALID_ARG;
    if (!pos && s->max_positions < s->T) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

template <typename T, bool INTER, bool PART>
void qk_launch2(int grid, cudaStream_t s, const QkParams& p, bool w) {
    if (w) qk_kernel<T, INTER, PART, true><<<grid, 256, 0, s>>>(p);
    else qk_kernel<T, INTER, PART, false><<<grid, 256, 0, s>>>(p);
}
template <typename T>
void qk_launch(int grid, cudaStream_t s, const QkParams& p, bool w) {
    const bool part = p.rd < p.d;
    if (p.inter) part ? qk_launch2<T, true, true>(grid, s, p, w) : qk_launch2<T, true, false>(grid, s, p, w);
    else part ? qk_launch2<T, false, true>(grid, s, p, w) : qk_launch2<T, false, false>(grid, s, p, w);
}
template <typename T, bool INTER, bool PART>
void qk_bwd_launch2(int grid, size_t smem, cudaStream_t s, const QkParams& p, bool w) {
    if (w) qk_bwd_kernel<T, INTER, PART, true><<<grid, 256, smem, s>>>(p);
    else qk_bwd_kernel<T, INTER, PART, false><<<grid, 256, smem, s>>>(p);
}
template <typename T>
void qk_bwd_launch(int grid, size_t smem, cudaStream_t s, const QkParams& p, bool w) {
    const bool part = p.rd < p.d;
    if (p.inter) part ? qk_bwd_launch2<T, true, true>(grid, smem, s, p, w) : qk_bwd_launch2<T, true, false>(grid, smem, s, p, w);
    else part ? qk_bwd_launch2<T, false, true>(grid, smem, s, p, w) : qk_bwd_launch2<T, false, false>(grid, smem, s, p, w);
}

// The gradient's items: a token with all its head passes where the tokens give every warp one, else
// as many passes as go together.
int qk_bwd_passes(const gdn_qk_shape* s, const QkParams& p) {
    const int most = p.pq > p.pk ? p.pq : p.pk;
    return s->T >= kSMs * 2 * 8 || most < 2 ? most : 2;
}
// CTAs of the gradient: one wave of two an SM (128 registers a thread), an item per warp at least.
int qk_bwd_ctas(const gdn_qk_shape* s) {
    const QkParams p = qk_params(s);
    const int passes = qk_bwd_passes(s, p), most = p.pq > p.pk ? p.pq : p.pk;
    const int64_t want = (s->T * ((most + passes - 1) / passes) + 7) / 8;
    return (int)(want < kSMs * 2 ? (want > 1 ? want : 1) : kSMs * 2);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_qk_norm_rope(const gdn_qk_shape* shape, const void* q, const void* k, const float* q_weight,
                                       const float* k_weight, const float* cos, const float* sin,
                                       const int32_t* positions, void* q_out, void* k_out, void* stream) {
    using namespace gdn;
    gdn_status st = check_qk(shape);
    if (st != GDN_OK) return st;
    if (shape->T == 0) return GDN_OK;
    const bool has_k = shape->HK > 0;
    if (!q || !q_out || (has_k && (!k || !k_out))) return GDN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) || !aligned16(k_weight))
        return GDN_ERR_INVALID_ARG;
    st = check_angles(shape, cos, sin, positions);
    if (st != GDN_OK) return st;
    if ((q_out == q && shape->ldq != (int64_t)shape->HQ * shape->d) || (has_k && k_out == k && shape->ldk != (int64_t)shape->HK * shape->d) ||
        (has_k && (q_out == k || k_out == q || q_out == k_out)))
        return GDN_ERR_INVALID_ARG;
    QkParams p = qk_params(shape);
    p.q = q, p.k = k, p.qw = q_weight, p.kw = k_weight, p.cos = cos, p.sin = sin, p.pos = positions;
    p.qo = q_out, p.ko = k_out;
    const int all = p.pq + p.pk;
    // A warp takes all the heads of a token where there are tokens for every SM's warps, else one pass each.
    p.passes = shape->T >= kSMs * 16 ? all : 1;
    p.items = p.T * ((all + p.passes - 1) / p.passes);
    const int64_t want = (p.items + 7) / 8;
    const int grid = (int)(want < kSMs * 16 ? want : kSMs * 16);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool w = q_weight || k_weight;
    if (shape->dtype == GDN_BF16) qk_launch<__nv_bfloat16>(grid, s, p, w);
    else qk_launch<float>(grid, s, p, w);
    return launch_status();
}

extern "C" size_t gdn_qk_norm_rope_bwd_workspace_size(const gdn_qk_shape* shape) {
    using namespace gdn;
    if (check_qk(shape) != GDN_OK) return 0;
    return (size_t)qk_bwd_ctas(shape) * 2 * shape->d * sizeof(float);
}

extern "C" gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_shape* shape, const void* q, const void* k,
                                           const float* q_weight, const float* k_weight, const float* cos,
                                           const float* sin, const int32_t* positions, const void* d_q_out,
                                           const void* d_k_out, void* dq, void* dk, int64_t lddq, int64_t lddk,
                                           float* dq_weight, float* dk_weight, void* workspace,
                                           size_t workspace_bytes, void* stream) {
    using namespace gdn;
    gdn_status st = check_qk(shape);
    if (st != GDN_OK) return st;
    const bool rows = shape->T > 0, has_k = shape->HK > 0;
    const int vn = shape->dtype == GDN_BF16 ? 8 : 4;
    const int64_t nq = (int64_t)shape->HQ * shape->d, nk = (int64_t)shape->HK * shape->d;
    if (rows && (!q || !d_q_out || !dq || (has_k && (!k || !d_k_out || !dk)))) return GDN_ERR_INVALID_ARG;
    if (lddq < nq || lddq % vn || (has_k && (lddk < nk || lddk % vn))) return GDN_ERR_INVALID_ARG;
    if ((dq_weight && !q_weight) || (dk_weight && (!k_weight || !has_k))) return GDN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(d_q_out) || !aligned16(d_k_out) || !aligned16(dq) || !aligned16(dk) ||
        !aligned16(q_weight) || !aligned16(k_weight) || !aligned4(dq_weight) || !aligned4(dk_weight))
        return GDN_ERR_INVALID_ARG;
    st = rows ? check_angles(shape, cos, sin, positions) : GDN_OK;
    if (st != GDN_OK) return st;
    if (rows && ((dq == d_q_out && lddq != nq) || (has_k && dk == d_k_out && lddk != nk) || dq == q || (has_k && (dk == k || dk == dq || dq == k || dk == q || dq == d_k_out || dk == d_q_out))))
        return GDN_ERR_INVALID_ARG;
    const bool sums = dq_weight || dk_weight;
    if (sums && (!workspace || !aligned16(workspace) || workspace_bytes < gdn_qk_norm_rope_bwd_workspace_size(shape)))
        return GDN_ERR_WORKSPACE;
    QkParams p = qk_params(shape);
    p.q = q, p.k = k, p.qw = q_weight, p.kw = k_weight, p.cos = cos, p.sin = sin, p.pos = positions;
    p.dqo = d_q_out, p.dko = d_k_out, p.qo = dq, p.ko = dk, p.lddq = lddq, p.lddk = lddk;
    p.part = sums ? static_cast<float*>(workspace) : nullptr;
    p.passes = qk_bwd_passes(shape, p);
    const int ctas = qk_bwd_ctas(shape);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = sums ? (size_t)(256 / p.lpr) * p.d * sizeof(float) : 0;
    const bool w = q_weight || k_weight;
    if (shape->dtype == GDN_BF16) qk_bwd_launch<__nv_bfloat16>(ctas, smem, s, p, w);
    else qk_bwd_launch<float>(ctas, smem, s, p, w);
    st = launch_status();
    if (st != GDN_OK || !sums) return st;
    qk_bwd_sum_kernel<<<dim3((unsigned)((p.d + 15) / 16), 2), 256, 0, s>>>(p.d, ctas, p.part, dq_weight, dk_weight);
    return launch_status();
}
