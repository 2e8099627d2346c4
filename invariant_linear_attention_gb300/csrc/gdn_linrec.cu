// gdn_linrec.cu -- the gated linear recurrence: prompts (and the trainer's forward), single tokens and
// the gradient.  The arithmetic is in gdn_linrec.cuh.
#include "gdn_async.cuh"
#include "gdn_host.h"
#include "gdn_linrec.cuh"

namespace gdn {
namespace {

using namespace linrec;

#ifndef LR_WORK
#define LR_WORK 256
#endif
#ifndef LR_AHEAD
#define LR_AHEAD 2
#endif
#ifndef LR_MINB
#define LR_MINB 2
#endif
// Prompts.  A CTA walks one sequence over CB channels in tiles of TT tokens.  Nearly all the work of a token does not
// depend on the one before it: only h <- a h + b does, 4 cycles a token.  So in step i
//   * the workers, a 16-byte chunk of one token each, finish tile i - 2 (gate, 16-byte stores of y) and prepare tile i
//     (a and b, to shared memory);
//   * the walkers, a lane a channel, walk tile i - 1 and leave h in b's place;
// and one barrier ends the step.  A worker reads the h of the very places that it then writes, so two buffers do.  Workers
// copy their own inputs asynchronously, AHEAD tiles ahead, and read back only what they copied themselves.
template <typename T, int CB>
struct FwdTile {
    static constexpr int VN = V16<T>::n, CH = CB / VN, WORK = LR_WORK, TT = WORK / CH, WALK = CB < 32 ? 32 : CB, NT = WORK + WALK;
    static constexpr int AHEAD = LR_AHEAD, ST = AHEAD + 1;
    float a[2][TT][CB], b[2][TT][CB];
    uint4 in[ST][4][WORK];  // x, a_gate, x_gate of a tile, z of the one two before
    float K[CB];
    // Channel c of row t lies at place(t, c): 16-byte pieces of neighbouring chunks side by side, and halves swapped in every
    // other row where a row is short, so that the workers' accesses (eight lanes at a time: one piece of eight chunks) meet no bank twice.
    static constexpr int PIECES = VN / 4;  // of a chunk
    static __device__ __forceinline__ int swap(int t) { return PIECES == 1 || CB > 32 ? 0 : CB == 32 ? t & 1 : (t >> 1) & 1; }
    static __device__ __forceinline__ int piece(int t, int ch, int e) { return ((e ^ swap(t)) * CH + ch) * 4; }
    static __device__ __forceinline__ int place(int t, int c) { return piece(t, c / VN, c % VN / 4) + c % 4; }
};

// All threads of the CTA meet, from whichever place in the code.
template <int THREADS>
__device__ __forceinline__ void step_end() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

template <typename T, int CB>
__global__ void __launch_bounds__(FwdTile<T, CB>::NT, LR_MINB) linrec_fwd_kernel(const __grid_constant__ Params p) {
    using F = FwdTile<T, CB>;
    constexpr int VN = F::VN, NP = VN / 2, CH = F::CH, TT = F::TT, WORK = F::WORK, AHEAD = F::AHEAD, ST = F::ST;
    extern __shared__ __align__(16) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const int blocks = (p.C + CB - 1) / CB, n = blockIdx.x / blocks, c0 = blockIdx.x % blocks * CB;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int tiles = (eos - bos + TT - 1) / TT;
    if (p.ap && threadIdx.x >= WORK && threadIdx.x - WORK < CB)
        sm.K[threadIdx.x - WORK] = c0 + (int)(threadIdx.x - WORK) < p.C ? rate_of(__ldg(p.ap + c0 + threadIdx.x - WORK), p.decay) : 0.f;
    __syncthreads();

    if (threadIdx.x < WORK) {
        const int tid = threadIdx.x, row = tid / CH, ch = tid % CH, c = c0 + ch * VN;
        const bool cok = c < p.C, gate = p.z != nullptr;
        float2 K[NP];
#pragma unroll
        for (int e = 0; e < NP; ++e) K[e] = make_float2(sm.K[ch * VN + 2 * e], sm.K[ch * VN + 2 * e + 1]);
        auto copy = [&](int i) {  // what step i needs
            uint4(&to)[4][WORK] = sm.in[i % ST];
            const int64_t t = (int64_t)bos + (int64_t)i * TT + row, tz = t - 2 * TT;
            if (t < eos && cok) {
                copy16_async(&to[0][tid], static_cast<const T*>(p.x) + t * p.ldx + c);
                copy16_async(&to[1][tid], static_cast<const T*>(p.ag) + t * p.lda + c);
                if (p.xg) copy16_async(&to[2][tid], static_cast<const T*>(p.xg) + t * p.ldg + c);
            }
            if (gate && tz >= bos && tz < eos && cok) copy16_async(&to[3][tid], static_cast<const T*>(p.z) + tz * p.ldz + c);
            copy_commit();
        };
        for (int i = 0; i < AHEAD; ++i) copy(i);
        for (int i = 0; i < tiles + 2; ++i) {
            copy(i + AHEAD);
            copy_wait<AHEAD>();
            const uint4(&in)[4][WORK] = sm.in[i % ST];
            float* ha = sm.a[i & 1][row];
            float* hb = sm.b[i & 1][row];
            const int64_t t = (int64_t)bos + (int64_t)i * TT + row, told = t - 2 * TT;
            if (told >= bos && told < eos && cok) {
                float2 h[NP];
#pragma unroll
                for (int e = 0; e < F::PIECES; ++e) {
                    const float4 v = *reinterpret_cast<const float4*>(hb + F::piece(row, ch, e));
                    h[2 * e] = make_float2(v.x, v.y), h[2 * e + 1] = make_float2(v.z, v.w);
                }
                if (gate) {
                    float2 z[NP];
                    unpack2(in[3][tid], z);
                    branch(p.act, z, h);
                }
                st16_stream(static_cast<T*>(p.y) + told * p.C + c, pack2(h));
            }
            if (t < eos) {
                float2 x[NP], ag[NP], xg[NP], a[NP], b[NP];
                unpack2(in[0][tid], x);
                unpack2(in[1][tid], ag);
                unpack2(in[2][tid], xg);
                steps(p, K, ag, xg, x, a, b);
#pragma unroll
                for (int e = 0; e < F::PIECES; ++e) {
                    *reinterpret_cast<float4*>(ha + F::piece(row, ch, e)) = make_float4(a[2 * e].x, a[2 * e].y, a[2 * e + 1].x, a[2 * e + 1].y);
                    *reinterpret_cast<float4*>(hb + F::piece(row, ch, e)) = make_float4(b[2 * e].x, b[2 * e].y, b[2 * e + 1].x, b[2 * e + 1].y);
                }
            }
            step_end<F::NT>();
        }
        copy_wait<0>();
        return;
    }

    const int cl = threadIdx.x - WORK, c = c0 + cl;
    const bool ok = cl < CB && c < p.C;
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    const bool has_slot = ok && slot >= 0 && slot < p.num_slots;
    float* st = p.state + (int64_t)slot * p.C + c;
    float h = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0) ? *st : 0.f;
    const int at[4] = {F::place(0, cl % CB), F::place(1, cl % CB), F::place(2, cl % CB), F::place(3, cl % CB)};
    for (int i = 0; i < tiles + 2; ++i) {
        const int len = i >= 1 ? min(TT, eos - bos - (i - 1) * TT) : 0;
        const float* a = sm.a[(i - 1) & 1][0];
        float* b = sm.b[(i - 1) & 1][0];
        constexpr int U = 16;
        int t = 0;
        if (len >= U) {  // the next 16 tokens' a and b are under way while 16 are walked
            float an[U], bn[U];
#pragma unroll
            for (int k = 0; k < U; ++k) an[k] = a[k * CB + at[k & 3]], bn[k] = b[k * CB + at[k & 3]];
            for (; t + U <= len; t += U) {
                float ak[U], bk[U];
#pragma unroll
                for (int k = 0; k < U; ++k) ak[k] = an[k], bk[k] = bn[k];
                if (t + 2 * U <= len) {
#pragma unroll
                    for (int k = 0; k < U; ++k) an[k] = a[(t + U + k) * CB + at[k & 3]], bn[k] = b[(t + U + k) * CB + at[k & 3]];
                }
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    h = __fmaf_rn(ak[k], h, bk[k]);
                    b[(t + k) * CB + at[k & 3]] = h;
                }
            }
        }
        for (; t < len; ++t) {
            h = __fmaf_rn(a[t * CB + at[t & 3]], h, b[t * CB + at[t & 3]]);
            b[t * CB + at[t & 3]] = h;
        }
        step_end<F::NT>();
    }
    if (has_slot) *st = h;
}

// Single tokens: a thread takes a chunk of channels over `rows` batch rows, so that it works out their rates once.
template <typename T>
__global__ void __launch_bounds__(128) linrec_update_kernel(const __grid_constant__ Params p, int rows) {
    constexpr int VN = V16<T>::n, NP = VN / 2;
    const int chunks = p.C / VN, blocks = (chunks + 127) / 128, ch = blockIdx.x % blocks * 128 + threadIdx.x, c = ch * VN;
    if (ch >= chunks) return;
    float2 K[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) K[e] = p.ap ? make_float2(rate_of(__ldg(p.ap + c + 2 * e), p.decay), rate_of(__ldg(p.ap + c + 2 * e + 1), p.decay)) : both(0.f);
    const int first = blockIdx.x / blocks * rows, last = min(first + rows, p.N);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t n = first; n < last; ++n) {
        const int slot = p.idx ? __ldg(p.idx + n) : (int)n;
        if (slot < 0 || slot >= p.num_slots) continue;
        float4* st = reinterpret_cast<float4*>(p.state + (int64_t)slot * p.C + c);
        const uint4 xr = ld16(static_cast<const T*>(p.x) + n * p.ldx + c), ar = ld16(static_cast<const T*>(p.ag) + n * p.lda + c);
        const uint4 gr = p.xg ? ld16(static_cast<const T*>(p.xg) + n * p.ldg + c) : none, zr = p.z ? ld16(static_cast<const T*>(p.z) + n * p.ldz + c) : none;
        float2 h[NP], x[NP], ag[NP], xg[NP], a[NP], b[NP];
#pragma unroll
        for (int e = 0; e < NP; e += 2) {
            const float4 v = st[e / 2];
            h[e] = make_float2(v.x, v.y), h[e + 1] = make_float2(v.z, v.w);
        }
        unpack2(xr, x);
        unpack2(ar, ag);
        unpack2(gr, xg);
        steps(p, K, ag, xg, x, a, b);
#pragma unroll
        for (int e = 0; e < NP; ++e) h[e] = __ffma2_rn(a[e], h[e], b[e]);
#pragma unroll
        for (int e = 0; e < NP; e += 2) st[e / 2] = make_float4(h[e].x, h[e].y, h[e + 1].x, h[e + 1].y);
        if (p.z) {
            float2 z[NP];
            unpack2(zr, z);
            branch(p.act, z, h);
        }
        st16(static_cast<T*>(p.y) + n * p.C + c, pack2(h));
    }
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
        const float2 K1[1] = {both(K)}, g1[1] = {both(ag)}, i1[1] = {both(xg)}, x1[1] = {both(x)};
        float2 a[1], b[1];
        steps(p, K1, g1, i1, x1, a, b);
        h = __fmaf_rn(a[0].x, h, b[0].x);
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
            const float2 w1[1] = {__fmul2_rn(both(K), r)};
            float2 a1[1], m1[1];
            decays(w1, a1, m1);
            w = w1[0], a = a1[0], m = m1[0];
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

#ifndef LR_CB
#define LR_CB 0
#endif
template <typename T, int CB>
gdn_status launch_fwd_of(cudaStream_t s, const Params& p) {
    using F = FwdTile<T, CB>;
    if (cudaFuncSetAttribute(linrec_fwd_kernel<T, CB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess) return GDN_ERR_CUDA;
    linrec_fwd_kernel<T, CB><<<(unsigned)((p.C + CB - 1) / CB) * (unsigned)p.N, F::NT, sizeof(F), s>>>(p);
    return launch_status();
}
template <typename T>
gdn_status launch_fwd(cudaStream_t s, const Params& p) {
    if (LR_CB == 16 || (LR_CB == 0 && (long long)((p.C + 31) / 32) * p.N <= kSMs / 2)) return launch_fwd_of<T, 16>(s, p);
    return launch_fwd_of<T, LR_CB ? LR_CB : 32>(s, p);
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
    return shape->dtype == GDN_BF16 ? launch_fwd<__nv_bfloat16>(s, p) : launch_fwd<float>(s, p);
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
    // as many rows a thread as leave every SM 16 CTAs
    const int blocks = (p.C / (shape->dtype == GDN_BF16 ? 8 : 4) + 127) / 128;
    const long long most = (long long)blocks * p.N / (kSMs * 16);
    const int rows = most < 1 ? 1 : most > 16 ? 16 : (int)most;
    const unsigned grid = (unsigned)blocks * (unsigned)((p.N + rows - 1) / rows);
    if (shape->dtype == GDN_BF16) linrec_update_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p, rows);
    else linrec_update_kernel<float><<<grid, 128, 0, s>>>(p, rows);
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
