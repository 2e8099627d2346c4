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
// groups and goes on to the token's other heads with the same cos and sin in registers.
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

// The pairs of a unit by its angles (back: by their negatives).  Halves: (a[e], b[e]); neighbours: (a[2e], a[2e+1]), then b's.
template <int VN>
__device__ __forceinline__ void rotate(float (&a)[VN], float (&b)[VN], const float (&cs)[VN], const float (&sn)[VN],
                                       bool inter, bool back) {
#pragma unroll
    for (int e = 0; e < VN; ++e) {
        const float s = back ? -sn[e] : sn[e];
        if (!inter) {
            const float u = a[e], v = b[e];
            a[e] = __fmaf_rn(u, cs[e], -__fmul_rn(v, s));
            b[e] = __fmaf_rn(v, cs[e], __fmul_rn(u, s));
        }
    }
    if (inter) {
#pragma unroll
        for (int e = 0; e < VN; ++e) {
            const float s = back ? -sn[e] : sn[e];
            float& u0 = e < VN / 2 ? a[(2 * e) % VN] : b[(2 * e) % VN];
            float& v0 = e < VN / 2 ? a[(2 * e + 1) % VN] : b[(2 * e + 1) % VN];
            const float u = u0, v = v0;
            u0 = __fmaf_rn(u, cs[e], -__fmul_rn(v, s));
            v0 = __fmaf_rn(v, cs[e], __fmul_rn(u, s));
        }
    }
}

template <int VN>
__device__ __forceinline__ void load_f(const float* p, bool ok, float other, float (&v)[VN]) {
#pragma unroll
    for (int e = 0; e < VN; e += 4) {
        const float4 u = ok ? __ldg(reinterpret_cast<const float4*>(p + e)) : make_float4(other, other, other, other);
        v[e] = u.x, v[e + 1] = u.y, v[e + 2] = u.z, v[e + 3] = u.w;
    }
}
template <int VN>
__device__ __forceinline__ void load_angles(const QkParams& p, int64_t pos, int u, bool rot, float (&cs)[VN], float (&sn)[VN]) {
#pragma unroll
    for (int e = 0; e < VN; ++e) {
        cs[e] = rot ? __ldg(p.cos + pos * (p.rd / 2) + u * VN + e) : 1.f;
        sn[e] = rot ? __ldg(p.sin + pos * (p.rd / 2) + u * VN + e) : 0.f;
    }
}

__device__ __forceinline__ float group_sum(float s, int lpr) {
    for (int off = 1; off < lpr; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

template <int VN>
__device__ __forceinline__ float squares(const float (&a)[VN], const float (&b)[VN]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < VN; ++e) s = __fmaf_rn(a[e], a[e], s);
#pragma unroll
    for (int e = 0; e < VN; ++e) s = __fmaf_rn(b[e], b[e], s);
    return s;
}

// The token's angle row, or -1 where it is skipped.
__device__ __forceinline__ int64_t angle_row(const QkParams& p, int64_t t) {
    if (p.rd == 0) return 0;
    const int64_t pos = p.pos ? (int64_t)__ldg(p.pos + t) : t;
    return pos >= 0 && pos < p.max_pos ? pos : -1;
}

template <typename T>
__global__ void __launch_bounds__(256) qk_kernel(const QkParams p) {
    constexpr int VN = V16<T>::n;
    const int lane = threadIdx.x & 31, u = lane & (p.lpr - 1), sub = lane / p.lpr, hpw = 32 / p.lpr;
    const Unit un = unit_of<VN>(u, p.d, p.rd, p.inter);
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int all = p.pq + p.pk, per = (all + p.passes - 1) / p.passes;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t it = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; it < p.items; it += nwarps) {
        const int64_t t = it / per;
        const int64_t row = angle_row(p, t);
        if (row < 0) continue;
        float cs[VN], sn[VN];
        load_angles<VN>(p, row, u, un.rot, cs, sn);
        const int first = (int)(it % per) * p.passes, last = min(first + p.passes, all);
        for (int ps = first; ps < last; ++ps) {
            const bool isq = ps < p.pq;
            const int h = (isq ? ps : ps - p.pq) * hpw + sub;
            const bool ok = h < (isq ? p.HQ : p.HK);
            const T* src = (isq ? static_cast<const T*>(p.q) + t * p.ldq : static_cast<const T*>(p.k) + t * p.ldk) + (int64_t)h * p.d;
            T* dst = (isq ? static_cast<T*>(p.qo) + t * p.HQ * p.d : static_cast<T*>(p.ko) + t * p.HK * p.d) + (int64_t)h * p.d;
            const float* w = isq ? p.qw : p.kw;
            float a[VN], b[VN], wa[VN], wb[VN];
            unpack(ok && un.has0 ? ld16_stream(src + un.e0) : none, a);
            unpack(ok && un.has1 ? ld16_stream(src + un.e1) : none, b);
            load_f<VN>(w + un.e0, w && un.has0, 1.f, wa);
            load_f<VN>(w + un.e1, w && un.has1, 1.f, wb);
            const float r = __frsqrt_rn(__fmaf_rn(group_sum(squares<VN>(a, b), p.lpr), p.c, p.eps));
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                a[e] = __fmul_rn(__fmul_rn(a[e], r), wa[e]);
                b[e] = __fmul_rn(__fmul_rn(b[e], r), wb[e]);
            }
            if (un.rot) rotate<VN>(a, b, cs, sn, p.inter, false);
            if (ok && un.has0) st16_stream(dst + un.e0, pack(a));
            if (ok && un.has1) st16_stream(dst + un.e1, pack(b));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) qk_bwd_kernel(const QkParams p) {
    constexpr int VN = V16<T>::n;
    extern __shared__ float acc[];  // [256 / lpr groups][d]
    const int lane = threadIdx.x & 31, u = lane & (p.lpr - 1), sub = lane / p.lpr, hpw = 32 / p.lpr;
    const Unit un = unit_of<VN>(u, p.d, p.rd, p.inter);
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {  // q, then k
        const int H = side ? p.HK : p.HQ, np = side ? p.pk : p.pq;
        const float* w = side ? p.kw : p.qw;
        const int64_t ld = side ? p.ldk : p.ldq, ldd = side ? p.lddk : p.lddq;
        const T* x = static_cast<const T*>(side ? p.k : p.q);
        const T* dout = static_cast<const T*>(side ? p.dko : p.dqo);
        T* dx = static_cast<T*>(side ? p.ko : p.qo);
        float wa[VN], wb[VN], sa[VN], sb[VN];
        load_f<VN>(w + un.e0, w && un.has0, 1.f, wa);
        load_f<VN>(w + un.e1, w && un.has1, 1.f, wb);
#pragma unroll
        for (int e = 0; e < VN; ++e) sa[e] = sb[e] = 0.f;
        for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < p.T; t += nwarps) {
            const int64_t row = angle_row(p, t);
            if (row < 0) continue;
            float cs[VN], sn[VN];
            load_angles<VN>(p, row, u, un.rot, cs, sn);
            for (int ps = 0; ps < np; ++ps) {
                const int h = ps * hpw + sub;
                const bool ok = h < H;
                const T* src = x + t * ld + (int64_t)h * p.d;
                const T* dsrc = dout + (t * H + h) * p.d;
                T* dst = dx + t * ldd + (int64_t)h * p.d;
                float a[VN], b[VN], ga[VN], gb[VN];
                unpack(ok && un.has0 ? ld16_stream(src + un.e0) : none, a);
                unpack(ok && un.has1 ? ld16_stream(src + un.e1) : none, b);
                unpack(ok && un.has0 ? ld16_stream(dsrc + un.e0) : none, ga);
                unpack(ok && un.has1 ? ld16_stream(dsrc + un.e1) : none, gb);
                const float r = __frsqrt_rn(__fmaf_rn(group_sum(squares<VN>(a, b), p.lpr), p.c, p.eps));
                if (un.rot) rotate<VN>(ga, gb, cs, sn, p.inter, true);
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    sa[e] = __fmaf_rn(__fmul_rn(a[e], r), ga[e], sa[e]);
                    sb[e] = __fmaf_rn(__fmul_rn(b[e], r), gb[e], sb[e]);
                    ga[e] = __fmul_rn(ga[e], wa[e]), gb[e] = __fmul_rn(gb[e], wb[e]);
                    dot = __fmaf_rn(ga[e], a[e], dot);
                    dot = __fmaf_rn(gb[e], b[e], dot);
                }
                dot = group_sum(dot, p.lpr);
                const float f = -__fmul_rn(__fmul_rn(__fmul_rn(r, r), __fmul_rn(r, p.c)), dot);
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    a[e] = __fmaf_rn(a[e], f, __fmul_rn(r, ga[e]));
                    b[e] = __fmaf_rn(b[e], f, __fmul_rn(r, gb[e]));
                }
                if (ok && un.has0) st16_stream(dst + un.e0, pack(a));
                if (ok && un.has1) st16_stream(dst + un.e1, pack(b));
            }
        }
        // the CTA's sum for the weight: its lane groups in ascending order
        if (w && p.part) {
            float* mine = acc + (int64_t)(threadIdx.x / p.lpr) * p.d;
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                if (un.has0) mine[un.e0 + e] = sa[e];
                if (un.has1) mine[un.e1 + e] = sb[e];
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

// dweight [d] of q (blockIdx.y 0) and k (1): a warp adds the CTAs' partials of one value, lane l
// those of CTAs l, l + 32, .. in order, then a butterfly.
__global__ void __launch_bounds__(256) qk_bwd_sum_kernel(int d, int ctas, const float* __restrict__ part,
                                                         float* __restrict__ dqw, float* __restrict__ dkw) {
    const int e = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, side = blockIdx.y;
    float* out = side ? dkw : dqw;
    if (e >= d || !out) return;
    float s = 0.f;
    for (int i = threadIdx.x & 31; i < ctas; i += 32) s = __fadd_rn(s, part[((int64_t)i * 2 + side) * d + e]);
    s = group_sum(s, 32);
    if ((threadIdx.x & 31) == 0) out[e] = s;
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
    if (!cos || !sin || !aligned4(cos) || !aligned4(sin) || !aligned4(pos)) return GDN_ERR_INVALID_ARG;
    if (!pos && s->max_positions < s->T) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// CTAs of the gradient: every SM several, a token per warp at least.
int qk_bwd_ctas(const gdn_qk_shape* s) {
    const int64_t want = (s->T + 7) / 8;
    return (int)(want < kSMs * 4 ? (want > 1 ? want : 1) : kSMs * 4);
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
    if (shape->dtype == GDN_BF16) qk_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else qk_kernel<float><<<grid, 256, 0, s>>>(p);
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
    const int ctas = qk_bwd_ctas(shape);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t smem = sums ? (size_t)(256 / p.lpr) * p.d * sizeof(float) : 0;
    if (shape->dtype == GDN_BF16) qk_bwd_kernel<__nv_bfloat16><<<ctas, 256, smem, s>>>(p);
    else qk_bwd_kernel<float><<<ctas, 256, smem, s>>>(p);
    st = launch_status();
    if (st != GDN_OK || !sums) return st;
    qk_bwd_sum_kernel<<<dim3((unsigned)((p.d + 7) / 8), 2), 256, 0, s>>>(p.d, ctas, p.part, dq_weight, dk_weight);
    return launch_status();
}
