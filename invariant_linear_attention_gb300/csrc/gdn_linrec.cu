// gdn_linrec.cu -- the gated linear recurrence: prompts (and the trainer's forward), single tokens and
// the gradient.  The arithmetic is in gdn_linrec.cuh.
#include "gdn_async.cuh"
#include "gdn_host.h"
#include "gdn_linrec.cuh"

namespace gdn {
namespace {

using namespace linrec;

#ifndef LR_SKIP
#define LR_SKIP 1
#endif
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
//   * the workers, each four tokens of two channels (fp32: of one), finish tile i - 2 (gate, stores of y) and prepare
//     tile i (a and b, to shared memory);
//   * the walkers, a lane a channel, walk tile i - 1 and leave h in b's place;
// and one barrier ends the step.  A worker reads the h of the very places that it then writes, so two buffers do.  The
// inputs arrive by asynchronous 16-byte copies, AHEAD tiles ahead.
template <typename T, int CB, int WORKERS, int TILES, bool APART>
struct FwdTile {
    static constexpr int VN = V16<T>::n, CH = CB / VN, WORK = WORKERS, TT = WORK / CH, WALK = CB < 32 ? 32 : CB, NT = WORK + WALK;
    static constexpr int LAUNCH = APART ? 32 * ((WORK / 32 + 2) / 3 * 4) + (WORK / 32 % 3 ? 32 * (WORK / 32 % 3 - 3) : 0) : NT;  // threads, with those that only keep their places
    static constexpr int AHEAD = TILES, ST = AHEAD + 1;
    static constexpr int W = VN / 4, P = CB / W;  // a worker's channels; workers of a token
    // Four tokens of a channel are 16 bytes, the walker's unit (with 4-byte loads its three a token took 14 cycles, not 4).
    // Even channels come first, then the odd ones: a worker's two are P units apart, and its neighbours' next to them.
    float4 a[2][TT / 4][CB], b[2][TT / 4][CB];
    // x, a_gate, x_gate of a tile, z of the one two before.  Rows shorter than 128 bytes share them; their order there goes
    // by the row's group of four too, so that a warp's workers, of several groups, meet no bank twice.
    uint4 in[ST][4][WORK];
    float K[CB];
    static constexpr int RS = 8 / CH;  // rows of 128 bytes
    static __device__ __forceinline__ int line(int t) { return (t & ~(RS - 1)) | ((t ^ (t >> 2)) & (RS - 1)); }
    static_assert(CH <= 8 && TT % 16 == 0, "rows of at most 128 bytes, tiles of whole walks");
};

// Shared memory in the order written: the compiler moves neither across the other.
__device__ __forceinline__ float4 ld_shared4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared4(uint32_t at, const float4& v) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
// All threads of the CTA meet, from whichever place in the code.
template <int THREADS>
__device__ __forceinline__ void step_end() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Four tokens of a worker's channels: values [token] of two channels (bf16), [pair of tokens] of one (fp32).
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
    static constexpr int NP = 4;
    static __device__ __forceinline__ void load(const uint4* in, const int (&at)[4], float2 (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t u = reinterpret_cast<const uint32_t*>(in)[at[j]];
            v[j] = make_float2(bf_lo(u), bf_hi(u));
        }
    }
    static __device__ __forceinline__ void put(float4* to, int P, const float2 (&v)[4]) {
        to[0] = make_float4(v[0].x, v[1].x, v[2].x, v[3].x), to[P] = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
    }
    static __device__ __forceinline__ void get(const float4* from, int P, float2 (&v)[4]) {
        const float4 x = from[0], y = from[P];
        v[0] = make_float2(x.x, y.x), v[1] = make_float2(x.y, y.y), v[2] = make_float2(x.z, y.z), v[3] = make_float2(x.w, y.w);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* y, int64_t ld, int rows, const float2 (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < rows) *reinterpret_cast<uint32_t*>(y + j * ld) = bf_pack(v[j].x, v[j].y);
    }
};
template <>
struct Four<float> {
    static constexpr int NP = 2;
    static __device__ __forceinline__ void load(const uint4* in, const int (&at)[4], float2 (&v)[2]) {
        const float* f = reinterpret_cast<const float*>(in);
        v[0] = make_float2(f[at[0]], f[at[1]]), v[1] = make_float2(f[at[2]], f[at[3]]);
    }
    static __device__ __forceinline__ void put(float4* to, int, const float2 (&v)[2]) { to[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
    static __device__ __forceinline__ void get(const float4* from, int, float2 (&v)[2]) {
        const float4 x = from[0];
        v[0] = make_float2(x.x, x.y), v[1] = make_float2(x.z, x.w);
    }
    static __device__ __forceinline__ void store(float* y, int64_t ld, int rows, const float2 (&v)[2]) {
        const float f[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < rows) y[j * ld] = f[j];
    }
};

template <typename T, typename F, int CB, int CTAS>
__global__ void __launch_bounds__(F::LAUNCH, CTAS) linrec_fwd_kernel(const __grid_constant__ Params p) {
    using Q = Four<T>;
    constexpr int VN = F::VN, NP = Q::NP, CH = F::CH, TT = F::TT, WORK = F::WORK, AHEAD = F::AHEAD, ST = F::ST, P = F::P;
    extern __shared__ __align__(16) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const int blocks = (p.C + CB - 1) / CB, n = blockIdx.x / blocks, c0 = blockIdx.x % blocks * CB;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int tiles = (eos - bos + TT - 1) / TT;
    if (p.ap && threadIdx.x < CB) sm.K[threadIdx.x] = c0 + (int)threadIdx.x < p.C ? rate_of(__ldg(p.ap + c0 + threadIdx.x), p.decay) : 0.f;

    if (threadIdx.x >= F::WALK) {
        int tid = threadIdx.x - F::WALK;
        if (F::LAUNCH > F::NT) {  // every fourth warp shares the walker's scheduler
            if (threadIdx.x / 32 % 4 == 0) return;
            tid = threadIdx.x - 32 * (threadIdx.x / 128 + 1);
        }
        const bool gate = p.z != nullptr;
        // its copies: a chunk of row tid / CH
        const int row = tid / CH, slot = F::line(row) * CH + tid % CH, cc = c0 + tid % CH * VN;
        int left = cc < p.C ? eos - bos - row : 0;  // rows from the next copy's on; below 1: none to copy
        const T* px = static_cast<const T*>(p.x) + (int64_t)(bos + row) * p.ldx + cc;
        const T* pa = static_cast<const T*>(p.ag) + (int64_t)(bos + row) * p.lda + cc;
        const T* pg = p.xg ? static_cast<const T*>(p.xg) + (int64_t)(bos + row) * p.ldg + cc : nullptr;
        const T* pz = gate ? static_cast<const T*>(p.z) + (int64_t)(bos + row) * p.ldz + cc : nullptr;
        int stage = 0, zleft = left, behind = 2;
        auto copy = [&] {  // what the next step that has no copies yet needs
            uint4(&to)[4][WORK] = sm.in[stage];
            stage = stage + 1 == ST ? 0 : stage + 1;
            if (left > 0) {
                copy16_async(&to[0][slot], px);
                copy16_async(&to[1][slot], pa);
                if (p.xg) copy16_async(&to[2][slot], pg);
            }
            px += (int64_t)TT * p.ldx, pa += (int64_t)TT * p.lda, pg += (int64_t)TT * p.ldg, left -= TT;
            if (behind > 0) {
                --behind;
            } else {
                if (gate && zleft > 0) copy16_async(&to[3][slot], pz);
                pz += (int64_t)TT * p.ldz, zleft -= TT;
            }
            copy_commit();
        };
        // its work: tokens 4 q .. of channels c ..
        const int q = tid / P, pr = tid % P, c = c0 + pr * F::W;
        const bool cok = c < p.C;
        int at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) at[j] = F::line(4 * q + j) * P + pr;  // in units of a worker's channels
        for (int i = 0; i < AHEAD; ++i) copy();
        copy_wait<AHEAD - 1>();
        step_end<F::NT>();
        float2 K[NP];
        const float2 k2 = F::W == 2 ? make_float2(sm.K[2 * pr], sm.K[2 * pr + 1]) : both(sm.K[pr]);
#pragma unroll
        for (int e = 0; e < NP; ++e) K[e] = k2;
        const bool far = any_far(K);
        T* y = static_cast<T*>(p.y) + (int64_t)(bos + 4 * q) * p.C + c;
        int rows = cok ? eos - bos - 4 * q : 0, old = 0;  // tokens from this step's on, and from the one's two before
        for (int i = 0, in = 0; i < tiles + 2; ++i) {
            copy();
            const uint4(&from)[4][WORK] = sm.in[in];
            in = in + 1 == ST ? 0 : in + 1;
            if (i == 2) old = cok ? eos - bos - 4 * q : 0;
            if (old > 0) {
                float2 h[NP];
                Q::get(&sm.b[i & 1][q][pr], P, h);
                if (gate) {
                    float2 z[NP];
                    Q::load(from[3], at, z);
                    branch(p.act, z, h);
                }
                Q::store(y, p.C, old, h);
                y += (int64_t)TT * p.C, old -= TT;
            }
            if (rows > 0) {
                float2 x[NP], ag[NP], xg[NP], a[NP], b[NP];
                Q::load(from[0], at, x);
                Q::load(from[1], at, ag);
                Q::load(from[2], at, xg);
                steps(p, far, K, ag, xg, x, a, b);
                Q::put(&sm.a[i & 1][q][pr], P, a);
                Q::put(&sm.b[i & 1][q][pr], P, b);
                rows -= TT;
            }
            copy_wait<AHEAD - 1>();
            step_end<F::NT>();
        }
        copy_wait<0>();
        return;
    }

    const int pos = threadIdx.x % CB, c = c0 + (F::W == 2 ? pos % P * 2 + pos / P : pos);  // neighbouring lanes, neighbouring units
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);  // (with 16 channels a second half of the lanes does the same)
    const bool has_slot = c < p.C && slot >= 0 && slot < p.num_slots;
    float* st = p.state + (int64_t)slot * p.C + c;
    float h = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0) ? *st : 0.f;
    step_end<F::NT>();
    for (int i = 0; i < tiles + 2; ++i) {
        const int len = i >= 1 ? min(TT, eos - bos - (i - 1) * TT) : 0;
        const uint32_t a = smem_u32(&sm.a[(i - 1) & 1][0][pos]), b = smem_u32(&sm.b[(i - 1) & 1][0][pos]);
        constexpr int U = 4;  // units walked while the next ones' loads are under way; at the end those read on into what follows, unused
        constexpr uint32_t step = CB * 16;
        const int units = len > 0 ? len / 4 : 0;
        int u = 0;
        auto walk4 = [&](const float4& av, const float4& bv, uint32_t to) {
            float4 o;
            h = o.x = __fmaf_rn(av.x, h, bv.x), h = o.y = __fmaf_rn(av.y, h, bv.y), h = o.z = __fmaf_rn(av.z, h, bv.z), h = o.w = __fmaf_rn(av.w, h, bv.w);
            st_shared4(to, o);
        };
        if (units >= 2 * U) {
            float4 ak[U], bk[U], an[U], bn[U];
            auto load = [&](int from, float4(&av)[U], float4(&bv)[U]) {
#pragma unroll
                for (int k = 0; k < U; ++k) av[k] = ld_shared4(a + (from + k) * step), bv[k] = ld_shared4(b + (from + k) * step);
            };
            load(0, ak, bk);
            for (; u + 2 * U <= units; u += 2 * U) {
                load(u + U, an, bn);
#pragma unroll
                for (int k = 0; k < U; ++k) walk4(ak[k], bk[k], b + (u + k) * step);
                load(u + 2 * U, ak, bk);
#pragma unroll
                for (int k = 0; k < U; ++k) walk4(an[k], bn[k], b + (u + U + k) * step);
            }
        }
        for (; u < units; ++u) walk4(ld_shared4(a + u * step), ld_shared4(b + u * step), b + u * step);
        if (4 * u < len) {
            const float4 av = ld_shared4(a + u * step), bv = ld_shared4(b + u * step);
            const float af[3] = {av.x, av.y, av.z}, bf[3] = {bv.x, bv.y, bv.z};
            float o[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (4 * u + k < len) h = o[k] = __fmaf_rn(af[k], h, bf[k]);
            st_shared4(b + u * step, make_float4(o[0], o[1], o[2], 0.f));
        }
        step_end<F::NT>();
    }
    if (has_slot && threadIdx.x < CB) *st = h;
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
    const bool far = any_far(K);
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
        steps(p, far, K, ag, xg, x, a, b);
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
        steps(p, true, K1, g1, i1, x1, a, b);
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
            decays(true, w1, a1, m1);
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
#ifndef LR_WORK2
#define LR_WORK2 512
#endif
#ifndef LR_AHEAD2
#define LR_AHEAD2 4
#endif
template <typename T, int CB, int WORKERS, int TILES, int CTAS, bool APART>
gdn_status launch_fwd_of(cudaStream_t s, const Params& p) {
    using F = FwdTile<T, CB, WORKERS, TILES, APART>;
    if (cudaFuncSetAttribute(linrec_fwd_kernel<T, F, CB, CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess) return GDN_ERR_CUDA;
    linrec_fwd_kernel<T, F, CB, CTAS><<<(unsigned)((p.C + CB - 1) / CB) * (unsigned)p.N, F::LAUNCH, sizeof(F), s>>>(p);
    return launch_status();
}
template <typename T>
gdn_status launch_fwd(cudaStream_t s, const Params& p) {
    if (LR_CB == 16 || (LR_CB == 0 && (long long)((p.C + 31) / 32) * p.N <= kSMs / 2)) return launch_fwd_of<T, 16, LR_WORK2, LR_AHEAD2, 1, LR_SKIP != 0>(s, p);
    return launch_fwd_of<T, 32, LR_WORK, LR_AHEAD, LR_MINB, false>(s, p);
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
