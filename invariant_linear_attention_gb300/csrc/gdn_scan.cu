// gdn_scan.cu -- the selective state space scan: prompts (and the trainer's forward) and
// single tokens.  The arithmetic is in gdn_scan.cuh.
#include "gdn_host.h"
#include "gdn_scan.cuh"

namespace gdn {
namespace {

using namespace scan;

// One lane's sums of L tokens over its own states, added over the L lanes of its channel:
// lane j ends with token j's sum.  Each level keeps half of the tokens and hands the others
// to the neighbour that keeps them, L - 1 shuffles in all; the additions are those of a
// butterfly (neighbours, then pairs of neighbours, ..).
template <int L>
__device__ __forceinline__ float scatter_sum(float (&s)[L], int j) {
#pragma unroll
    for (int off = 1, n = L; off < L; off <<= 1, n >>= 1) {
        const bool up = j & off;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? s[2 * i + 1] : s[2 * i], give = up ? s[2 * i] : s[2 * i + 1];
            s[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, off));
        }
    }
    return s[0];
}

// Prompts.  A CTA walks one sequence over CB channels, a lane 8 states of one channel (L = S / 8
// lanes a channel).  Per tile of TT tokens the threads first share the work per (token, channel),
// 16 bytes of x, dt and z each: d = softplus(dt + bias) and d x go to shared memory for the
// lanes, the next tile's loads are issued, the lanes walk the tile and leave sum_s h C in
// shared memory, and the threads add D x, apply the gate and store 16 bytes.
template <typename T, int S>
struct FwdTile {
    static constexpr int L = S / 8, CB = 128 / L, TT = 16, VN = V16<T>::n;
    static constexpr int CH = CB / VN;                        // 16-byte chunks of a row
    static constexpr int NV = (TT * CH + 127) / 128;          // of x (dt, z) per thread and tile
    static constexpr int BCH = S / VN;                        // chunks of a row of B (C)
    static constexpr int NB = (2 * TT * BCH + 127) / 128;     // of B and C per thread and tile
    // {d, d x} of channel c at c float2s plus one 16-byte gap per 16 channels: the chunk-wise
    // stores and the lanes' loads are both free of bank conflicts.
    static constexpr int ROW = CB + (CB / 16) * 2;            // float2s per token
    static constexpr int YROW = CB + (L > 1 ? 32 / L : 0);    // the lanes' stores of L tokens miss each other's banks
    alignas(16) float2 d[TT][ROW];
    alignas(16) float y[TT][YROW];
    alignas(16) float b[2][TT][S];
    alignas(16) float D[CB];
    alignas(16) float bias[CB];
};

template <typename T, int S>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const Params p) {
    using F = FwdTile<T, S>;
    constexpr int L = F::L, CB = F::CB, TT = F::TT, VN = F::VN, CH = F::CH, NV = F::NV, BCH = F::BCH, NB = F::NB;
    __shared__ __align__(16) F sm;
    const int tid = threadIdx.x;
    const int nb = p.bpg * p.G;
    const int n = blockIdx.x / nb, blk = blockIdx.x % nb;
    const int g = blk / p.bpg, cg0 = (blk % p.bpg) * CB, c0 = g * p.CG + cg0;
    const int j = tid % L, cl = tid / L;
    const bool ok = cg0 + cl < p.CG;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    const bool has_slot = slot >= 0 && slot < p.num_slots;
    const bool use_init = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0);

    for (int c = tid; c < CB; c += 128) {
        const bool in = cg0 + c < p.CG;
        sm.D[c] = in && p.D ? __ldg(p.D + c0 + c) : 0.f;
        sm.bias[c] = in && p.bias ? __ldg(p.bias + c0 + c) : 0.f;
    }
    float2 A2[4], h[4];
    const int64_t own = ok ? (int64_t)(c0 + cl) * S + 8 * j : 0;
    float* st = p.state + (int64_t)slot * p.C * S + own;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float2 t[2];
        load4(p.A_log + own + 4 * i, t);
        A2[2 * i] = make_float2(a_log2(t[0].x), a_log2(t[0].y));
        A2[2 * i + 1] = make_float2(a_log2(t[1].x), a_log2(t[1].y));
        const float4 u = use_init ? *reinterpret_cast<const float4*>(st + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
        h[2 * i] = make_float2(u.x, u.y), h[2 * i + 1] = make_float2(u.z, u.w);
    }
    const T* x = static_cast<const T*>(p.x) + c0;
    const T* dt = static_cast<const T*>(p.dt) + c0;
    const T* z = static_cast<const T*>(p.z) + c0;
    const T* Bg = static_cast<const T*>(p.B) + (int64_t)g * S;
    const T* Cg = static_cast<const T*>(p.Cm) + (int64_t)g * S;
    T* y = static_cast<T*>(p.y) + c0;
    const bool gate = p.z != nullptr, sp = p.softplus != 0;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);

    uint4 rx[NV], rd[NV], rz[NV], rb[NB];
    auto load = [&](int t0) {
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int v = tid + 128 * r, tt = v / CH, c = (v % CH) * VN;
            const int64_t t = t0 + tt;
            const bool in = tt < TT && t < eos && cg0 + c < p.CG;
            rx[r] = in ? ld16_stream(x + t * p.ldx + c) : none;
            rd[r] = in ? ld16_stream(dt + t * p.lddt + c) : none;
            rz[r] = in && gate ? ld16_stream(z + t * p.ldz + c) : none;
        }
#pragma unroll
        for (int r = 0; r < NB; ++r) {
            const int v = tid + 128 * r, which = v / (TT * BCH), w = v % (TT * BCH), tt = w / BCH;
            const int64_t t = t0 + tt;
            rb[r] = none;
            if (which < 2 && t < eos)
                rb[r] = ld16(which ? Cg + t * p.ldC + (w % BCH) * VN : Bg + t * p.ldB + (w % BCH) * VN);
        }
    };
    load(bos);
    __syncthreads();
    for (int t0 = bos; t0 < eos; t0 += TT) {
        uint4 cx[NV], cz[NV];
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int v = tid + 128 * r, tt = v / CH, c = (v % CH) * VN;
            cx[r] = rx[r], cz[r] = rz[r];
            if (tt < TT) {
                float xv[VN], dv[VN];
                unpack(rx[r], xv);
                unpack(rd[r], dv);
                float4* to = reinterpret_cast<float4*>(&sm.d[tt][c + (c / 16) * 2]);
#pragma unroll
                for (int e = 0; e < VN; e += 2) {
                    const float2 b2 = *reinterpret_cast<const float2*>(&sm.bias[c + e]);
                    const float d0 = step_of(dv[e], b2.x, sp), d1 = step_of(dv[e + 1], b2.y, sp);
                    to[e / 2] = make_float4(d0, __fmul_rn(d0, xv[e]), d1, __fmul_rn(d1, xv[e + 1]));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < NB; ++r) {
            const int v = tid + 128 * r, which = v / (TT * BCH), w = v % (TT * BCH);
            if (which < 2) {
                float f[VN];
                unpack(rb[r], f);
                float4* to = reinterpret_cast<float4*>(&sm.b[which][w / BCH][(w % BCH) * VN]);
#pragma unroll
                for (int e = 0; e < VN; e += 4) to[e / 4] = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
        }
        __syncthreads();
        load(t0 + TT);
        const int len = min(TT, eos - t0);
        const float2* dp = &sm.d[0][cl + (cl / 16) * 2];
        auto token = [&](int tt) {
            const float2 d = dp[tt * F::ROW];
            const float4* b4 = reinterpret_cast<const float4*>(&sm.b[0][tt][8 * j]);
            const float4* c4 = reinterpret_cast<const float4*>(&sm.b[1][tt][8 * j]);
            const float2 d2 = make_float2(d.x, d.x), x2 = make_float2(d.y, d.y);
            float2 acc;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 b = b4[i], c = c4[i];
                advance(h[2 * i], A2[2 * i], d2, x2, make_float2(b.x, b.y));
                advance(h[2 * i + 1], A2[2 * i + 1], d2, x2, make_float2(b.z, b.w));
                acc = i ? __ffma2_rn(h[2 * i], make_float2(c.x, c.y), acc) : __fmul2_rn(h[0], make_float2(c.x, c.y));
                acc = __ffma2_rn(h[2 * i + 1], make_float2(c.z, c.w), acc);
            }
            return __fadd_rn(acc.x, acc.y);
        };
        if (len == TT) {
#pragma unroll (TT / L > 4 ? 2 : 1)
            for (int tt = 0; tt < TT; tt += L) {
                float s[L];
#pragma unroll
                for (int i = 0; i < L; ++i) s[i] = token(tt + i);
                sm.y[tt + j][cl] = scatter_sum<L>(s, j);
            }
        } else {
            for (int tt = 0; tt < len; ++tt) {
                float s = token(tt);
#pragma unroll
                for (int off = 1; off < L; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
                if (j == 0) sm.y[tt][cl] = s;
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int v = tid + 128 * r, tt = v / CH, c = (v % CH) * VN;
            if (tt < len && cg0 + c < p.CG) {
                float xv[VN], zv[VN], out[VN];
                unpack(cx[r], xv);
                unpack(cz[r], zv);
#pragma unroll
                for (int e = 0; e < VN; e += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(&sm.y[tt][c + e]);
                    const float4 D4 = *reinterpret_cast<const float4*>(&sm.D[c + e]);
                    out[e] = finish_y(s4.x, D4.x, xv[e]), out[e + 1] = finish_y(s4.y, D4.y, xv[e + 1]);
                    out[e + 2] = finish_y(s4.z, D4.z, xv[e + 2]), out[e + 3] = finish_y(s4.w, D4.w, xv[e + 3]);
                }
                if (gate) {
#pragma unroll
                    for (int e = 0; e < VN; ++e) out[e] = __fmul_rn(out[e], silu_fast(zv[e]));
                }
                st16_stream(y + (int64_t)(t0 + tt) * p.C + c, pack(out));
            }
        }
    }
    if (has_slot && ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4*>(st + 4 * i) = make_float4(h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
    }
}

template <typename T, int S>
__global__ void __launch_bounds__(128) scan_update_kernel(const Params p) {
    constexpr int L = S / 4, CB = 128 / L;
    const int nb = p.bpg * p.G;
    const int n = blockIdx.x / nb, blk = blockIdx.x % nb;
    const int g = blk / p.bpg, j = threadIdx.x % L;
    const int cg = (blk % p.bpg) * CB + threadIdx.x / L;
    const bool ok = cg < p.CG;
    const int c = g * p.CG + (ok ? cg : 0);
    const int slot = p.idx ? __ldg(p.idx + n) : n;
    if (slot < 0 || slot >= p.num_slots) return;
    float2 A2[2], h[2], b[2], cc[2];
    load4(p.A_log + (int64_t)c * S + 4 * j, A2);
    float* st = p.state + ((int64_t)slot * p.C + c) * S + 4 * j;
    const float4 u = *reinterpret_cast<const float4*>(st);
    h[0] = make_float2(u.x, u.y), h[1] = make_float2(u.z, u.w);
    const float xv = load1(static_cast<const T*>(p.x) + n * p.ldx + c);
    const float d = step_of(load1(static_cast<const T*>(p.dt) + n * p.lddt + c), p.bias ? __ldg(p.bias + c) : 0.f, p.softplus);
    const float dx = __fmul_rn(d, xv);
    load4(static_cast<const T*>(p.B) + n * p.ldB + (int64_t)g * S + 4 * j, b);
    load4(static_cast<const T*>(p.Cm) + n * p.ldC + (int64_t)g * S + 4 * j, cc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        advance(h[i], make_float2(a_log2(A2[i].x), a_log2(A2[i].y)), make_float2(d, d), make_float2(dx, dx), b[i]);
    float s = finish_y(sum_states4<L>(h, cc, j), p.D ? __ldg(p.D + c) : 0.f, xv);
    if (p.z) s = __fmul_rn(s, silu_fast(load1(static_cast<const T*>(p.z) + n * p.ldz + c)));
    if (!ok) return;
    if (j == 1) store1(static_cast<T*>(p.y) + (int64_t)n * p.C + c, s);
    *reinterpret_cast<float4*>(st) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
}

// Validation common to the two entry points; fills the parameters.
gdn_status prepare(const gdn_scan_shape* s, const void* x, const void* dt, const float* A_log, const void* B,
                   const void* Cm, const float* D, const void* z, const float* dt_bias, float* state,
                   const int32_t* idx, int num_slots, void* y, Params& p) {
    const bool rows = s->T_total > 0;
    if (!A_log || (rows && (!x || !dt || !B || !Cm || !y))) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(dt) || !aligned16(B) || !aligned16(Cm) || !aligned16(z) || !aligned16(y) ||
        !aligned16(A_log) || !aligned16(state) || !aligned4(D) || !aligned4(dt_bias) || !aligned4(idx))
        return GDN_ERR_INVALID_ARG;
    if (z && (s->ldz < s->C || s->ldz % (s->dtype == GDN_BF16 ? 8 : 4))) return GDN_ERR_INVALID_ARG;
    if (y && (y == x || y == dt || y == z || y == B || y == Cm)) return GDN_ERR_INVALID_ARG;
    if (state && (num_slots < 0 || (!idx && num_slots < s->N))) return GDN_ERR_INVALID_ARG;
    p = Params{};
    p.N = s->N, p.T = s->T_total, p.C = s->C, p.G = s->G, p.CG = s->C / s->G;
    p.softplus = s->dt_softplus;
    p.x = x, p.dt = dt, p.z = z, p.B = B, p.Cm = Cm;
    p.ldx = s->ldx, p.lddt = s->lddt, p.ldz = s->ldz, p.ldB = s->ldB, p.ldC = s->ldC;
    p.A_log = A_log, p.D = D, p.bias = dt_bias;
    p.state = state, p.idx = idx, p.num_slots = state ? num_slots : 0;
    p.y = y;
    return GDN_OK;
}

// K::cb(S): channels of a CTA.
template <template <typename, int> class K, typename T>
gdn_status by_states(int S, cudaStream_t s, Params& p) {
    const int cb = K<T, 8>::cb(S);
    p.bpg = (p.CG + cb - 1) / cb;
    const long long ctas = (long long)p.N * p.G * p.bpg;
    if (ctas >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    switch (S) {
        case 8: K<T, 8>::go((unsigned)ctas, s, p); break;
        case 16: K<T, 16>::go((unsigned)ctas, s, p); break;
        case 32: K<T, 32>::go((unsigned)ctas, s, p); break;
        case 64: K<T, 64>::go((unsigned)ctas, s, p); break;
        default: return GDN_ERR_UNSUPPORTED;
    }
    return launch_status();
}
template <typename T, int S>
struct FwdK {
    static int cb(int states) { return 128 / (states / 8); }
    static void go(unsigned grid, cudaStream_t s, const Params& p) { scan_fwd_kernel<T, S><<<grid, 128, 0, s>>>(p); }
};
template <typename T, int S>
struct UpdK {
    static int cb(int states) { return 128 / (states / 4); }
    static void go(unsigned grid, cudaStream_t s, const Params& p) { scan_update_kernel<T, S><<<grid, 128, 0, s>>>(p); }
};

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_selective_scan_fwd(const gdn_scan_shape* shape, const void* x, const void* dt,
                                             const float* A_log, const void* B, const void* Cm, const float* D,
                                             const void* z, const float* dt_bias, const int32_t* cu_seqlens,
                                             float* state, const int32_t* state_indices, int num_slots,
                                             const int32_t* has_initial_state, void* y, void* stream) {
    using namespace gdn;
    gdn_status st = check_scan(shape);
    if (st != GDN_OK) return st;
    if (shape->N == 0) return shape->T_total == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (!cu_seqlens || !aligned4(cu_seqlens) || !aligned4(has_initial_state)) return GDN_ERR_INVALID_ARG;
    scan::Params p;
    st = prepare(shape, x, dt, A_log, B, Cm, D, z, dt_bias, state, state_indices, num_slots, y, p);
    if (st != GDN_OK) return st;
    p.cu = cu_seqlens, p.has_init = has_initial_state;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return shape->dtype == GDN_BF16 ? by_states<FwdK, __nv_bfloat16>(shape->S, s, p)
                                    : by_states<FwdK, float>(shape->S, s, p);
}

extern "C" gdn_status gdn_selective_scan_update(const gdn_scan_shape* shape, const void* x, const void* dt,
                                                const float* A_log, const void* B, const void* Cm, const float* D,
                                                const void* z, const float* dt_bias, float* state,
                                                const int32_t* state_indices, int num_slots, void* y, void* stream) {
    using namespace gdn;
    gdn_status st = check_scan(shape);
    if (st != GDN_OK) return st;
    if (shape->T_total != shape->N) return GDN_ERR_INVALID_ARG;
    if (shape->N == 0) return GDN_OK;
    if (!state) return GDN_ERR_INVALID_ARG;
    scan::Params p;
    st = prepare(shape, x, dt, A_log, B, Cm, D, z, dt_bias, state, state_indices, num_slots, y, p);
    if (st != GDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return shape->dtype == GDN_BF16 ? by_states<UpdK, __nv_bfloat16>(shape->S, s, p)
                                    : by_states<UpdK, float>(shape->S, s, p);
}
