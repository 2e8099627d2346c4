// gdn_linrec.cu -- the gated linear recurrence: prompts (and the trainer's forward), single tokens and
// the gradient.  The arithmetic is in gdn_linrec.cuh.
#include "gdn_host.h"
#include "gdn_linrec.cuh"

namespace gdn {
namespace {

using namespace linrec;

// Prompts: a thread walks one channel of one sequence.
template <typename T>
__global__ void __launch_bounds__(128) linrec_fwd_kernel(const __grid_constant__ Params p) {
    const int blocks = (p.C + 127) / 128, n = blockIdx.x / blocks, c = blockIdx.x % blocks * 128 + threadIdx.x;
    if (c >= p.C) return;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    const bool has_slot = slot >= 0 && slot < p.num_slots;
    float* st = p.state + (int64_t)slot * p.C + c;
    float h = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0) ? *st : 0.f;
    const float K = p.ap ? rate_of(__ldg(p.ap + c), p.decay) : 0.f;
    for (int64_t t = bos; t < eos; ++t) {
        const float x = load1(static_cast<const T*>(p.x) + t * p.ldx + c), ag = load1(static_cast<const T*>(p.ag) + t * p.lda + c);
        const float xg = p.xg ? load1(static_cast<const T*>(p.xg) + t * p.ldg + c) : 0.f;
        float2 a, b;
        step2(p, both(K), both(ag), both(xg), both(x), a, b);
        h = __fmaf_rn(a.x, h, b.x);
        float y = h;
        if (p.z) y = __fmul_rn(h, act2(p.act, both(load1(static_cast<const T*>(p.z) + t * p.ldz + c))).x);
        store1(static_cast<T*>(p.y) + t * p.C + c, y);
    }
    if (has_slot) *st = h;
}

// Single tokens: a thread one channel of one sequence.
template <typename T>
__global__ void __launch_bounds__(128) linrec_update_kernel(const __grid_constant__ Params p) {
    const int blocks = (p.C + 127) / 128, c = blockIdx.x % blocks * 128 + threadIdx.x;
    const int64_t n = blockIdx.x / blocks;
    if (c >= p.C) return;
    const int slot = p.idx ? __ldg(p.idx + n) : (int)n;
    if (slot < 0 || slot >= p.num_slots) return;
    float* st = p.state + (int64_t)slot * p.C + c;
    const float K = p.ap ? rate_of(__ldg(p.ap + c), p.decay) : 0.f;
    const float x = load1(static_cast<const T*>(p.x) + n * p.ldx + c), ag = load1(static_cast<const T*>(p.ag) + n * p.lda + c);
    const float xg = p.xg ? load1(static_cast<const T*>(p.xg) + n * p.ldg + c) : 0.f;
    float2 a, b;
    step2(p, both(K), both(ag), both(xg), both(x), a, b);
    const float h = __fmaf_rn(a.x, *st, b.x);
    *st = h;
    float y = h;
    if (p.z) y = __fmul_rn(h, act2(p.act, both(load1(static_cast<const T*>(p.z) + n * p.ldz + c))).x);
    store1(static_cast<T*>(p.y) + n * p.C + c, y);
}

// Gradient: a thread one channel of one sequence, forward with every state to the workspace, then back.
//     e = dy act(z),  G_t = e_t + a_{t+1} G_{t+1},  dx = G s p,  dx_gate = G s x p (1 - p),  dz = dy h act'(z)
//     dL/du k = G (a h_{t-1} k - v k a^2 / s) with u = -w, k = u (or a_gate's slope 1 - a of log a):
//     da_gate that times 1 - r (or as it is), da_param its sum over the tokens times sigmoid(a_param) decay / K
struct GradParams {
    Params p;
    const void* dy;
    const float *h0, *dhT;
    void *dx, *da, *dg, *dz;
    float *dap, *dh0, *hs, *part;
};
template <typename T>
__global__ void __launch_bounds__(128) linrec_bwd_kernel(const __grid_constant__ GradParams q) {
    const Params& p = q.p;
    const int blocks = (p.C + 127) / 128, n = blockIdx.x / blocks, c = blockIdx.x % blocks * 128 + threadIdx.x;
    if (c >= p.C) return;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const float K = p.ap ? rate_of(__ldg(p.ap + c), p.decay) : 0.f;
    const int64_t own = (int64_t)n * p.C + c;
    const float h0 = q.h0 ? q.h0[own] : 0.f;
    float h = h0;
    for (int64_t t = bos; t < eos; ++t) {
        const float x = load1(static_cast<const T*>(p.x) + t * p.ldx + c), ag = load1(static_cast<const T*>(p.ag) + t * p.lda + c);
        const float xg = p.xg ? load1(static_cast<const T*>(p.xg) + t * p.ldg + c) : 0.f;
        float2 a, b;
        step2(p, both(K), both(ag), both(xg), both(x), a, b);
        h = __fmaf_rn(a.x, h, b.x);
        q.hs[t * p.C + c] = h;
    }
    float g = q.dhT ? q.dhT[own] : 0.f, sum = 0.f;
    for (int64_t t = eos - 1; t >= bos; --t) {
        const float x = load1(static_cast<const T*>(p.x) + t * p.ldx + c), ag = load1(static_cast<const T*>(p.ag) + t * p.lda + c);
        const float xg = p.xg ? load1(static_cast<const T*>(p.xg) + t * p.ldg + c) : 0.f;
        const float dy = load1(static_cast<const T*>(q.dy) + t * p.C + c);
        h = q.hs[t * p.C + c];
        const float old = t > bos ? q.hs[(t - 1) * p.C + c] : h0;
        float2 e, a, m, ep;
        const float2 r = sigmoid2(both(ag), e), r1 = rest2(e, r);
        float2 w = both(0.f);
        if (p.ap) {
            w = __fmul2_rn(both(K), r);
            decay2(w, a, m);
        } else {
            a = r, m = r1;
        }
        const float k = p.ap ? -w.x : m.x;
        float s = 1.f, kappa = 0.f;
        if (p.scale == GDN_SCALE_SQRT) {
            const float t2 = rest_of_square(a, m).x;
            s = sqrt_approx(t2);
            kappa = t2 > 0.f ? k * a.x * a.x * rsqrt_approx(t2) : 0.f;
        } else if (p.scale == GDN_SCALE_LINEAR) {
            s = m.x, kappa = k * a.x;
        }
        const float2 pg = p.xg ? sigmoid2(both(xg), ep) : both(1.f);
        const float v = x * pg.x;
        float ge = dy;
        if (p.z) {
            float2 slope;
            const float f = act2(p.act, both(load1(static_cast<const T*>(p.z) + t * p.ldz + c)), slope).x;
            store1(static_cast<T*>(q.dz) + t * p.C + c, dy * h * slope.x);
            ge = dy * f;
        }
        g = g + ge;
        const float dv = g * s;
        store1(static_cast<T*>(q.dx) + t * p.C + c, dv * pg.x);
        if (p.xg) store1(static_cast<T*>(q.dg) + t * p.C + c, dv * v * rest2(ep, pg).x);
        const float d = g * (a.x * old * k - v * kappa);
        store1(static_cast<T*>(q.da) + t * p.C + c, p.ap ? d * r1.x : d);
        sum += d;
        g = a.x * g;
    }
    if (q.dh0) q.dh0[own] = g;
    if (q.part) q.part[own] = sum;
}
__global__ void __launch_bounds__(128) linrec_param_kernel(int N, int C, float decay, const float* __restrict__ ap,
                                                           const float* __restrict__ part, float* __restrict__ out) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= C) return;
    float s = 0.f;
    for (int n = 0; n < N; ++n) s += part[(int64_t)n * C + c];
    const float v = __ldg(ap + c), K = rate_of(v, decay), sp = 1.f / (1.f + expf(-v));
    out[c] = K > 0.f ? s * (decay * sp / K) : 0.f;
}

gdn_status check_linrec(const gdn_linrec_shape* s, bool param, bool gate, bool z) {
    if (!s) return GDN_ERR_INVALID_ARG;
    if (s->N < 0 || s->T_total < 0 || s->C <= 0) return GDN_ERR_INVALID_ARG;
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (s->scale < GDN_SCALE_SQRT || s->scale > GDN_SCALE_ONE) return GDN_ERR_UNSUPPORTED;
    if (z && s->activation != GDN_ACT_SILU && s->activation != GDN_ACT_GELU) return GDN_ERR_UNSUPPORTED;
    if (param && !(s->decay > 0.f && s->decay <= FLT_MAX)) return GDN_ERR_INVALID_ARG;
    const int vn = s->dtype == GDN_BF16 ? 8 : 4;
    if (s->C % vn) return GDN_ERR_UNSUPPORTED;
    // CTAs are numbered, and states per sequence indexed, in 31 bits
    if (s->T_total > INT_MAX - 256 || (long long)s->N * s->C >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    if (s->ldx < s->C || s->lda < s->C || (gate && s->ldg < s->C) || (z && s->ldz < s->C)) return GDN_ERR_INVALID_ARG;
    if (s->ldx % vn || s->lda % vn || (gate && s->ldg % vn) || (z && s->ldz % vn)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Validation common to the three entry points; fills the parameters.
gdn_status prepare(const gdn_linrec_shape* s, const void* x, const void* ag, const float* ap, const void* xg, const void* z, Params& p) {
    gdn_status st = check_linrec(s, ap, xg, z);
    if (st != GDN_OK) return st;
    if (s->T_total > 0 && (!x || !ag)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(ag) || !aligned16(ap) || !aligned16(xg) || !aligned16(z)) return GDN_ERR_INVALID_ARG;
    p = Params{};
    p.N = s->N, p.T = s->T_total, p.C = s->C, p.scale = s->scale, p.act = s->activation, p.decay = s->decay;
    p.x = x, p.ag = ag, p.xg = xg, p.z = z, p.ap = ap;
    p.ldx = s->ldx, p.lda = s->lda, p.ldg = s->ldg, p.ldz = s->ldz;
    return GDN_OK;
}
gdn_status pool(Params& p, float* state, const int32_t* idx, int num_slots, void* y) {
    if (!aligned16(state) || !aligned4(idx) || !aligned16(y) || (p.T > 0 && !y)) return GDN_ERR_INVALID_ARG;
    if (y && (y == p.x || y == p.ag || y == p.xg || y == p.z)) return GDN_ERR_INVALID_ARG;
    if (state && (num_slots < 0 || (!idx && num_slots < p.N))) return GDN_ERR_INVALID_ARG;
    p.state = state, p.idx = idx, p.num_slots = state ? num_slots : 0, p.y = y;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_linear_recurrence_fwd(const gdn_linrec_shape* shape, const void* x, const void* a_gate,
                                                const float* a_param, const void* x_gate, const void* z,
                                                const int32_t* cu_seqlens, float* state, const int32_t* state_indices,
                                                int num_slots, const int32_t* has_initial_state, void* y, void* stream) {
    using namespace gdn;
    Params p;
    gdn_status st = prepare(shape, x, a_gate, a_param, x_gate, z, p);
    if (st == GDN_OK) st = pool(p, state, state_indices, num_slots, y);
    if (st != GDN_OK) return st;
    if (p.N == 0) return p.T == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (!cu_seqlens || !aligned4(cu_seqlens) || !aligned4(has_initial_state)) return GDN_ERR_INVALID_ARG;
    p.cu = cu_seqlens, p.has_init = has_initial_state;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)((p.C + 127) / 128) * (unsigned)p.N;
    if (shape->dtype == GDN_BF16) linrec_fwd_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p);
    else linrec_fwd_kernel<float><<<grid, 128, 0, s>>>(p);
    return launch_status();
}

extern "C" gdn_status gdn_linear_recurrence_update(const gdn_linrec_shape* shape, const void* x, const void* a_gate,
                                                   const float* a_param, const void* x_gate, const void* z, float* state,
                                                   const int32_t* state_indices, int num_slots, void* y, void* stream) {
    using namespace gdn;
    Params p;
    gdn_status st = prepare(shape, x, a_gate, a_param, x_gate, z, p);
    if (st == GDN_OK) st = pool(p, state, state_indices, num_slots, y);
    if (st != GDN_OK) return st;
    if (p.T != p.N) return GDN_ERR_INVALID_ARG;
    if (p.N == 0) return GDN_OK;
    if (!state) return GDN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)((p.C + 127) / 128) * (unsigned)p.N;
    if (shape->dtype == GDN_BF16) linrec_update_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p);
    else linrec_update_kernel<float><<<grid, 128, 0, s>>>(p);
    return launch_status();
}

extern "C" size_t gdn_linear_recurrence_bwd_workspace_size(const gdn_linrec_shape* shape) {
    using namespace gdn;
    if (check_linrec(shape, false, false, false) != GDN_OK) return 0;
    return ((size_t)shape->T_total + shape->N) * shape->C * sizeof(float);
}

extern "C" gdn_status gdn_linear_recurrence_bwd(const gdn_linrec_shape* shape, const void* x, const void* a_gate,
                                                const float* a_param, const void* x_gate, const void* z,
                                                const int32_t* cu_seqlens, const float* init_state, const void* d_y,
                                                const float* d_final_state, void* dx, void* da_gate, float* da_param,
                                                void* dx_gate, void* dz, float* d_init_state, void* workspace,
                                                size_t workspace_bytes, void* stream) {
    using namespace gdn;
    GradParams q{};
    gdn_status st = prepare(shape, x, a_gate, a_param, x_gate, z, q.p);
    if (st != GDN_OK) return st;
    const Params& p = q.p;
    const bool rows = p.T > 0;
    if (rows && (!d_y || !dx || !da_gate || (x_gate && !dx_gate) || (z && !dz))) return GDN_ERR_INVALID_ARG;
    if (!aligned16(d_y) || !aligned16(dx) || !aligned16(da_gate) || !aligned16(dx_gate) || !aligned16(dz) || !aligned16(init_state) ||
        !aligned16(d_final_state) || !aligned16(d_init_state) || !aligned16(da_param))
        return GDN_ERR_INVALID_ARG;
    if (da_param && !a_param) return GDN_ERR_INVALID_ARG;
    if (d_init_state && (d_init_state == init_state || d_init_state == d_final_state)) return GDN_ERR_INVALID_ARG;
    if (p.N == 0 && rows) return GDN_ERR_INVALID_ARG;
    if (p.N > 0 && (!cu_seqlens || !aligned4(cu_seqlens))) return GDN_ERR_INVALID_ARG;
    const void* in[] = {x, a_gate, x_gate, z, d_y};
    const void* out[] = {dx, da_gate, x_gate ? dx_gate : nullptr, z ? dz : nullptr};
    for (int i = 0; i < 4; ++i) {
        for (const void* v : in)
            if (out[i] && out[i] == v) return GDN_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return GDN_ERR_INVALID_ARG;
    }
    if (p.N > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < gdn_linear_recurrence_bwd_workspace_size(shape)))
        return GDN_ERR_WORKSPACE;
    q.p.cu = cu_seqlens;
    q.dy = d_y, q.h0 = init_state, q.dhT = d_final_state, q.dx = dx, q.da = da_gate, q.dg = dx_gate, q.dz = dz;
    q.dap = da_param, q.dh0 = d_init_state;
    q.hs = static_cast<float*>(workspace), q.part = da_param ? q.hs + (size_t)p.T * p.C : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned blocks = (unsigned)((p.C + 127) / 128);
    if (p.N > 0) {
        if (shape->dtype == GDN_BF16) linrec_bwd_kernel<__nv_bfloat16><<<blocks * p.N, 128, 0, s>>>(q);
        else linrec_bwd_kernel<float><<<blocks * p.N, 128, 0, s>>>(q);
        st = launch_status();
        if (st != GDN_OK) return st;
    }
    if (!da_param) return GDN_OK;
    linrec_param_kernel<<<blocks, 128, 0, s>>>(p.N, p.C, p.decay, a_param, q.part, da_param);
    return launch_status();
}
