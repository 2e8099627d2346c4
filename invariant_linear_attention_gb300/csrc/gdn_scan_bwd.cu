// gdn_scan_bwd.cu -- gradient of the selective scan.  With e = d_y silu(z) and g the gradient
// with respect to h:
//
//     g_t = e_t Cm_t + a_{t+1} g_{t+1}      (from d_final_state behind the last token)
//     dC = sum_c e h,  dB = sum_c g d x,  u = sum_s g B,  w = g a h_{t-1}
//     dx = d u + D e,  dd = x u + sum_s w A,  ddt = dd sigmoid,  dz = d_y (y / silu) silu'
//     dA_log = A sum_t w d,  dD = sum_t e x,  ddt_bias = sum_t ddt,  d_init_state = a_0 g_0
//
// First the states at every kChunk-th token (the forward recurrence without its outputs), then
// the chunks of a sequence last to first: a chunk's states are recomputed into registers and
// walked backwards.  The sums over channels leave one partial per channel block, the sums over
// tokens one per sequence; two small kernels add those up in order.
#include "gdn_host.h"
#include "gdn_scan.cuh"

namespace gdn {
namespace {

using namespace scan;

constexpr int kChunk = 8;

struct BwdParams {
    Params f;
    const float *h0, *dhT;
    const void* dy;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *dbias, *dh0;
    float *ckpt, *bc, *pA, *pD, *pb;
};

// Chunk k of sequence n is number cu[n] / kChunk + n + k: never two on one number.
__device__ __forceinline__ int64_t chunk_base(int bos, int n) { return (int64_t)(bos / kChunk) + n; }

struct Lane {
    int n, g, j, c, blk;
    bool ok;
};
template <int S>
__device__ __forceinline__ Lane lane_of(const Params& p) {
    constexpr int L = S / 4, CB = 128 / L;
    const int nb = p.bpg * p.G;
    Lane l;
    l.n = blockIdx.x / nb, l.blk = blockIdx.x % nb;
    l.g = l.blk / p.bpg, l.j = threadIdx.x % L;
    const int cg = (l.blk % p.bpg) * CB + threadIdx.x / L;
    l.ok = cg < p.CG;
    l.c = l.g * p.CG + (l.ok ? cg : 0);
    return l;
}

__device__ __forceinline__ void load_state(const float* p, float2 (&h)[2]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    h[0] = make_float2(u.x, u.y), h[1] = make_float2(u.z, u.w);
}
__device__ __forceinline__ void store_state(float* p, const float2 (&h)[2]) {
    *reinterpret_cast<float4*>(p) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
}

template <typename T, int S>
__global__ void __launch_bounds__(128) scan_states_kernel(const BwdParams q) {
    const Params& p = q.f;
    const Lane l = lane_of<S>(p);
    int bos, eos;
    bounds(p.cu, l.n, p.T, bos, eos);
    if (!l.ok) return;
    float2 A2[2], h[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    load4(p.A_log + (int64_t)l.c * S + 4 * l.j, A2);
#pragma unroll
    for (int i = 0; i < 2; ++i) A2[i] = make_float2(a_log2(A2[i].x), a_log2(A2[i].y));
    if (q.h0) load_state(q.h0 + ((int64_t)l.n * p.C + l.c) * S + 4 * l.j, h);
    const float bias = p.bias ? __ldg(p.bias + l.c) : 0.f;
    const T* x = static_cast<const T*>(p.x) + l.c;
    const T* dt = static_cast<const T*>(p.dt) + l.c;
    const T* B = static_cast<const T*>(p.B) + (int64_t)l.g * S + 4 * l.j;
    float* out = q.ckpt + (chunk_base(bos, l.n) * p.C + l.c) * S + 4 * l.j;
    for (int t = bos; t < eos; ++t) {
        if ((t - bos) % kChunk == 0) {
            store_state(out, h);
            out += (int64_t)p.C * S;
        }
        const float d = step_of(both(load1(dt + t * p.lddt)), both(bias), p.softplus).x;
        const float dx = __fmul_rn(d, load1(x + t * p.ldx));
        float2 b[2];
        load4(B + t * p.ldB, b);
#pragma unroll
        for (int i = 0; i < 2; ++i) advance(h[i], A2[i], make_float2(d, d), make_float2(dx, dx), b[i]);
    }
}

template <int L>
__device__ __forceinline__ float sum_lanes(float s) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}
template <int L>
__device__ __forceinline__ float sum_channels(float s) {
#pragma unroll
    for (int off = L; off < 32; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

template <typename T, int S>
__global__ void __launch_bounds__(128) scan_bwd_kernel(const BwdParams q) {
    constexpr int L = S / 4;
    __shared__ float sums[4][kChunk][2][S];  // per warp: dB and dC of the chunk's tokens
    const Params& p = q.f;
    const Lane l = lane_of<S>(p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int bos, eos;
    bounds(p.cu, l.n, p.T, bos, eos);
    float2 A2[2], A[2], G[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    load4(p.A_log + (int64_t)l.c * S + 4 * l.j, A2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        A[i] = make_float2(-expf(A2[i].x), -expf(A2[i].y));
        A2[i] = make_float2(a_log2(A2[i].x), a_log2(A2[i].y));
    }
    const int64_t so = ((int64_t)l.n * p.C + l.c) * S + 4 * l.j;
    if (q.dhT) load_state(q.dhT + so, G);
    float2 dA[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    float dD = 0.f, db = 0.f;
    const float bias = p.bias ? __ldg(p.bias + l.c) : 0.f, D = p.D ? __ldg(p.D + l.c) : 0.f;
    const T* x = static_cast<const T*>(p.x) + l.c;
    const T* dt = static_cast<const T*>(p.dt) + l.c;
    const T* z = p.z ? static_cast<const T*>(p.z) + l.c : nullptr;
    const T* dy = static_cast<const T*>(q.dy) + l.c;
    const T* B = static_cast<const T*>(p.B) + (int64_t)l.g * S + 4 * l.j;
    const T* Cm = static_cast<const T*>(p.Cm) + (int64_t)l.g * S + 4 * l.j;
    const int chunks = (eos - bos + kChunk - 1) / kChunk;
    for (int k = chunks - 1; k >= 0; --k) {
        const int t0 = bos + k * kChunk, len = min(kChunk, eos - t0);
        float2 h[2], ah[kChunk][2], a[kChunk][2];
        load_state(q.ckpt + ((chunk_base(bos, l.n) + k) * p.C + l.c) * S + 4 * l.j, h);
        float ysum[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            if (i >= len) break;
            const int t = t0 + i;
            const float d = step_of(both(load1(dt + t * p.lddt)), both(bias), p.softplus).x;
            const float dx = __fmul_rn(d, load1(x + t * p.ldx));
            float2 b[2], cc[2];
            load4(B + t * p.ldB, b);
            load4(Cm + t * p.ldC, cc);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 e = __fmul2_rn(make_float2(d, d), A2[m]);
                a[i][m] = make_float2(ex2(e.x), ex2(e.y));
                ah[i][m] = __fmul2_rn(a[i][m], h[m]);
                h[m] = __ffma2_rn(make_float2(dx, dx), b[m], ah[i][m]);
            }
            ysum[i] = z ? sum_states4<L>(h, cc, l.j) : 0.f;
        }
#pragma unroll
        for (int i = kChunk - 1; i >= 0; --i) {
            if (i >= len) continue;
            const int t = t0 + i;
            const float xv = load1(x + t * p.ldx);
            float sig = 1.f, d = __fadd_rn(load1(dt + t * p.lddt), bias);
            if (p.softplus) {
                float2 u;
                const float2 v = both(d);
                d = softplus2(v, u).x;
                sig = sigmoid2(v, u).x;
            }
            const float dx = __fmul_rn(d, xv);
            const float dyv = l.ok ? load1(dy + (int64_t)t * p.C) : 0.f;
            float e = dyv;
            if (z) {
                const float zv = load1(z + t * p.ldz), s = rcp_approx(__fadd_rn(1.f, __expf(-zv)));
                e = __fmul_rn(dyv, __fmul_rn(zv, s));
                const float ds = __fmul_rn(s, __fmaf_rn(zv, __fsub_rn(1.f, s), 1.f));
                if (l.ok && l.j == 1)
                    store1(static_cast<T*>(q.dz) + (int64_t)t * p.C + l.c, __fmul_rn(__fmul_rn(dyv, __fmaf_rn(D, xv, ysum[i])), ds));
            }
            float2 b[2], cc[2];
            load4(B + t * p.ldB, b);
            load4(Cm + t * p.ldC, cc);
            float2 u = make_float2(0.f, 0.f), v = u;
            const float2 e2 = make_float2(e, e), d2 = make_float2(d, d), dx2 = make_float2(dx, dx);
            float2 sb[2], sc[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 ht = __ffma2_rn(dx2, b[m], ah[i][m]);
                const float2 gt = __ffma2_rn(e2, cc[m], G[m]);
                u = __ffma2_rn(gt, b[m], u);
                const float2 w = __fmul2_rn(gt, ah[i][m]);
                v = __ffma2_rn(w, A[m], v);
                dA[m] = __ffma2_rn(w, d2, dA[m]);
                G[m] = __fmul2_rn(a[i][m], gt);
                sb[m] = l.ok ? __fmul2_rn(gt, dx2) : make_float2(0.f, 0.f);
                sc[m] = l.ok ? __fmul2_rn(ht, e2) : make_float2(0.f, 0.f);
            }
            const float us = sum_lanes<L>(__fadd_rn(u.x, u.y)), vs = sum_lanes<L>(__fadd_rn(v.x, v.y));
            const float ddt = __fmul_rn(__fmaf_rn(xv, us, vs), sig);
            dD = __fmaf_rn(e, xv, dD);
            db = __fadd_rn(db, ddt);
            if (l.ok && l.j == 0) {
                store1(static_cast<T*>(q.dx) + (int64_t)t * p.C + l.c, __fmaf_rn(d, us, __fmul_rn(D, e)));
                store1(static_cast<T*>(q.ddt) + (int64_t)t * p.C + l.c, ddt);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float v0 = sum_channels<L>(sb[m].x), v1 = sum_channels<L>(sb[m].y);
                const float v2 = sum_channels<L>(sc[m].x), v3 = sum_channels<L>(sc[m].y);
                if (lane < L) {
                    sums[warp][i][0][4 * l.j + 2 * m] = v0, sums[warp][i][0][4 * l.j + 2 * m + 1] = v1;
                    sums[warp][i][1][4 * l.j + 2 * m] = v2, sums[warp][i][1][4 * l.j + 2 * m + 1] = v3;
                }
            }
        }
        __syncthreads();
        for (int f = threadIdx.x; f < len * 2 * S; f += 128) {
            const float* r = &sums[0][0][0][0] + f;
            constexpr int W = kChunk * 2 * S;
            q.bc[((int64_t)l.blk * p.T + t0) * 2 * S + f] = __fadd_rn(__fadd_rn(r[0], r[W]), __fadd_rn(r[2 * W], r[3 * W]));
        }
        __syncthreads();
    }
    if (!l.ok) return;
    if (q.dh0) store_state(q.dh0 + so, G);
#pragma unroll
    for (int m = 0; m < 2; ++m) dA[m] = __fmul2_rn(dA[m], A[m]);
    store_state(q.pA + so, dA);
    if (l.j == 0) {
        q.pD[(int64_t)l.n * p.C + l.c] = dD;
        q.pb[(int64_t)l.n * p.C + l.c] = db;
    }
}

// dB and dC of every covered token: the channel blocks' partials of its group in order.
template <typename T, int S>
__global__ void __launch_bounds__(256) scan_bc_kernel(const BwdParams q) {
    const Params& p = q.f;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, per = (int64_t)p.G * 2 * S;
    const int end = max(0, min(__ldg(p.cu + p.N), p.T));
    const int64_t t = i / per;
    if (t >= end) return;
    const int g = (int)(i % per) / (2 * S), s = (int)(i % (2 * S));
    float sum = 0.f;
    for (int b = 0; b < p.bpg; ++b) sum = __fadd_rn(sum, q.bc[(((int64_t)g * p.bpg + b) * p.T + t) * 2 * S + s]);
    T* out = static_cast<T*>(s < S ? q.dB : q.dC);
    store1(out + (t * p.G + g) * S + (s < S ? s : s - S), sum);
}

// dA_log [C, S], dD, ddt_bias [C]: the sequences' partials in order.
__global__ void __launch_bounds__(256) scan_params_kernel(int N, int C, int S, const float* __restrict__ pA, const float* __restrict__ pD,
                                                          const float* __restrict__ pb, float* __restrict__ dA, float* __restrict__ dD,
                                                          float* __restrict__ db) {
    const int64_t nA = (int64_t)C * S, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= nA + 2 * C) return;
    const float* src = i < nA ? pA + i : i < nA + C ? pD + (i - nA) : pb + (i - nA - C);
    float* dst = i < nA ? dA + i : i < nA + C ? (dD ? dD + (i - nA) : nullptr) : (db ? db + (i - nA - C) : nullptr);
    if (!dst) return;
    float s = 0.f;
    for (int n = 0; n < N; ++n) s = __fadd_rn(s, src[n * (i < nA ? nA : C)]);
    *dst = s;
}

struct Layout {
    size_t ckpt, bc, pA, pD, pb, total;  // offsets in floats
    int bpg;
};
Layout layout(const gdn_scan_shape* s) {
    const int cb = 128 / (s->S / 4), cg = s->C / s->G;
    Layout l;
    l.bpg = (cg + cb - 1) / cb;
    const size_t cs = (size_t)s->C * s->S;
    l.ckpt = 0;
    l.bc = l.ckpt + ((size_t)s->T_total / kChunk + s->N) * cs;
    l.pA = l.bc + (size_t)s->G * l.bpg * s->T_total * 2 * s->S;
    l.pD = l.pA + s->N * cs;
    l.pb = l.pD + (size_t)s->N * s->C;
    l.total = l.pb + (size_t)s->N * s->C;
    return l;
}

template <typename T, int S>
gdn_status launch(cudaStream_t s, const BwdParams& q) {
    const Params& p = q.f;
    const long long ctas = (long long)p.N * p.G * p.bpg, bc = ((long long)p.T * p.G * 2 * S + 255) / 256;
    if (ctas >= (1LL << 31) || bc >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    scan_states_kernel<T, S><<<(unsigned)ctas, 128, 0, s>>>(q);
    scan_bwd_kernel<T, S><<<(unsigned)ctas, 128, 0, s>>>(q);
    if (bc) scan_bc_kernel<T, S><<<(unsigned)bc, 256, 0, s>>>(q);
    scan_params_kernel<<<(unsigned)(((int64_t)p.C * (S + 2) + 255) / 256), 256, 0, s>>>(p.N, p.C, S, q.pA, q.pD, q.pb, q.dA, q.dD, q.dbias);
    return launch_status();
}
template <typename T>
gdn_status by_states(int S, cudaStream_t s, const BwdParams& q) {
    switch (S) {
        case 8: return launch<T, 8>(s, q);
        case 16: return launch<T, 16>(s, q);
        case 32: return launch<T, 32>(s, q);
        case 64: return launch<T, 64>(s, q);
    }
    return GDN_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace gdn

extern "C" size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_shape* shape) {
    using namespace gdn;
    if (check_scan(shape) != GDN_OK) return 0;
    return layout(shape).total * sizeof(float);
}

extern "C" gdn_status gdn_selective_scan_bwd(const gdn_scan_shape* shape, const void* x, const void* dt,
                                             const float* A_log, const void* B, const void* Cm, const float* D,
                                             const void* z, const float* dt_bias, const int32_t* cu_seqlens,
                                             const float* init_state, const void* d_y, const float* d_final_state,
                                             void* dx, void* ddt, float* dA_log, void* dB, void* dC, float* dD,
                                             void* dz, float* ddt_bias, float* d_init_state, void* workspace,
                                             size_t workspace_bytes, void* stream) {
    using namespace gdn;
    gdn_status st = check_scan(shape);
    if (st != GDN_OK) return st;
    const bool rows = shape->T_total > 0;
    if (rows && shape->N == 0) return GDN_ERR_INVALID_ARG;
    if (!A_log || !cu_seqlens || !dA_log || (rows && (!x || !dt || !B || !Cm || !d_y || !dx || !ddt || !dB || !dC || (z && !dz))))
        return GDN_ERR_INVALID_ARG;
    for (const void* v : {x, dt, B, Cm, z, d_y, (const void*)A_log, (const void*)init_state, (const void*)d_final_state,
                          (const void*)dx, (const void*)ddt, (const void*)dB, (const void*)dC, (const void*)dz,
                          (const void*)dA_log, (const void*)d_init_state})
        if (!aligned16(v)) return GDN_ERR_INVALID_ARG;
    for (const void* v : {(const void*)D, (const void*)dt_bias, (const void*)cu_seqlens, (const void*)dD, (const void*)ddt_bias})
        if (!aligned4(v)) return GDN_ERR_INVALID_ARG;
    if (z && (shape->ldz < shape->C || shape->ldz % (shape->dtype == GDN_BF16 ? 8 : 4))) return GDN_ERR_INVALID_ARG;
    for (const void* o : {(const void*)dx, (const void*)ddt, (const void*)dB, (const void*)dC, z ? (const void*)dz : nullptr})
        for (const void* v : {x, dt, B, Cm, z, d_y})
            if (o && o == v) return GDN_ERR_INVALID_ARG;
    if (d_init_state && (d_init_state == init_state || d_init_state == d_final_state)) return GDN_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < gdn_selective_scan_bwd_workspace_size(shape))
        return GDN_ERR_WORKSPACE;
    const Layout l = layout(shape);
    float* w = static_cast<float*>(workspace);
    BwdParams q{};
    scan::Params& p = q.f;
    p.N = shape->N, p.T = shape->T_total, p.C = shape->C, p.G = shape->G, p.CG = shape->C / shape->G, p.bpg = l.bpg;
    p.softplus = shape->dt_softplus;
    p.x = x, p.dt = dt, p.z = z, p.B = B, p.Cm = Cm;
    p.ldx = shape->ldx, p.lddt = shape->lddt, p.ldz = shape->ldz, p.ldB = shape->ldB, p.ldC = shape->ldC;
    p.A_log = A_log, p.D = D, p.bias = dt_bias, p.cu = cu_seqlens;
    q.h0 = init_state, q.dhT = d_final_state, q.dy = d_y;
    q.dx = dx, q.ddt = ddt, q.dz = dz, q.dB = dB, q.dC = dC;
    q.dA = dA_log, q.dD = dD, q.dbias = ddt_bias, q.dh0 = d_init_state;
    q.ckpt = w + l.ckpt, q.bc = w + l.bc, q.pA = w + l.pA, q.pD = w + l.pD, q.pb = w + l.pb;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (shape->N == 0) {  // no tokens, no sequences: the sums are empty
        scan_params_kernel<<<(unsigned)(((int64_t)p.C * (shape->S + 2) + 255) / 256), 256, 0, s>>>(0, p.C, shape->S, q.pA, q.pD, q.pb, q.dA, q.dD, q.dbias);
        return launch_status();
    }
    return shape->dtype == GDN_BF16 ? by_states<__nv_bfloat16>(shape->S, s, q) : by_states<float>(shape->S, s, q);
}
