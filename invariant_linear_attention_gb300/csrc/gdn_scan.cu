// gdn_scan.cu -- the selective state space scan: prompts (and the trainer's forward) and
// single tokens.  The arithmetic is in gdn_scan.cuh.
#include "gdn_host.h"
#include "gdn_scan.cuh"

namespace gdn {
namespace {

using namespace scan;

// A lane holds 4 states of a channel, S / 4 lanes a channel.
template <typename T, int S>
__global__ void __launch_bounds__(128) scan_fwd_kernel(const Params p) {
    constexpr int L = S / 4, CB = 128 / L;
    const int nb = p.bpg * p.G;
    const int n = blockIdx.x / nb, blk = blockIdx.x % nb;
    const int g = blk / p.bpg, j = threadIdx.x % L;
    const int cg = (blk % p.bpg) * CB + threadIdx.x / L;
    const bool ok = cg < p.CG;
    const int c = g * p.CG + (ok ? cg : 0);
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    const bool has_slot = slot >= 0 && slot < p.num_slots;
    const bool use_init = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0);
    float2 A2[2], h[2];
    load4(p.A_log + (int64_t)c * S + 4 * j, A2);
#pragma unroll
    for (int i = 0; i < 2; ++i) A2[i] = make_float2(a_log2(A2[i].x), a_log2(A2[i].y));
    float* st = p.state + ((int64_t)slot * p.C + c) * S + 4 * j;
    h[0] = h[1] = make_float2(0.f, 0.f);
    if (use_init) {
        const float4 u = *reinterpret_cast<const float4*>(st);
        h[0] = make_float2(u.x, u.y), h[1] = make_float2(u.z, u.w);
    }
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f, D = p.D ? __ldg(p.D + c) : 0.f;
    const T* x = static_cast<const T*>(p.x) + c;
    const T* dt = static_cast<const T*>(p.dt) + c;
    const T* z = p.z ? static_cast<const T*>(p.z) + c : nullptr;
    const T* B = static_cast<const T*>(p.B) + (int64_t)g * S + 4 * j;
    const T* Cm = static_cast<const T*>(p.Cm) + (int64_t)g * S + 4 * j;
    T* y = static_cast<T*>(p.y) + c;
    for (int t = bos; t < eos; ++t) {
        const float xv = load1(x + t * p.ldx);
        const float d = step_of(load1(dt + t * p.lddt), bias, p.softplus);
        const float dx = __fmul_rn(d, xv);
        float2 b[2], cc[2];
        load4(B + t * p.ldB, b);
        load4(Cm + t * p.ldC, cc);
#pragma unroll
        for (int i = 0; i < 2; ++i) advance(h[i], A2[i], make_float2(d, d), make_float2(dx, dx), b[i]);
        float s = finish_y(sum_states4<L>(h, cc, j), D, xv);
        if (z) s = __fmul_rn(s, silu_fast(load1(z + t * p.ldz)));
        if (ok && j == 1) store1(y + (int64_t)t * p.C, s);
    }
    if (has_slot && ok) *reinterpret_cast<float4*>(st) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
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

template <template <typename, int> class K, typename T>
gdn_status by_states(int S, cudaStream_t s, Params& p) {
    const int cb = 128 / (S / 4);
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
    static void go(unsigned grid, cudaStream_t s, const Params& p) { scan_fwd_kernel<T, S><<<grid, 128, 0, s>>>(p); }
};
template <typename T, int S>
struct UpdK {
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
