// gdn_scan.cuh -- the selective scan's per-element arithmetic, shared by the prompt, single
// token and gradient kernels so that they agree bit for bit.
//
//     d = softplus(dt + bias),  a = exp(d A),  h <- a h + (d x) B,  y = sum_s h C
//
// with A = -exp(A_log) held as A log2(e), so that a is one product and one hardware exponential.
// A channel's states are summed in this fixed tree: per 8 consecutive states one packed
// (even, odd) chain in ascending order, then even + odd; the 8-state sums as a balanced binary
// tree over neighbours.  How many of its states a thread holds (4 or 8 and up) is free.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gdn_scan.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace scan {

// A log2(e) of one state from its A_log.  Past fp32's range (A_log > 88.3) the largest finite value stands
// for it: any step that is not 0 still forgets such a state, but 0 times it (a step of 0, a tile's
// padding, the gradient of what was forgotten) is 0 and not NaN.
__device__ __forceinline__ float a_log2(float A_log) {
    const float a = __fmul_rn(-expf(A_log), kLog2e);
    return a < -FLT_MAX ? -FLT_MAX : a;
}

// softplus(v) = max(v, 0) + log(1 + u), u = e^-|v| in (0, 1], with log(1 + u) = 2 artanh(w),
// w = u / (2 + u) <= 1/3: relative accuracy is kept for the small steps of strongly negative v,
// which log of a rounded 1 + u would lose.  artanh(w) / w is a polynomial of degree 4 in w^2
// (Chebyshev interpolation on [0, 1/9], its constant term put to 1; error 8e-9).  Two values at a time, in packed operations.
// `u` is left for the derivative.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 softplus2(const float2& v, float2& u) {
    const float2 m = make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f));
    u = make_float2(ex2(__fmul_rn(fabsf(v.x), -kLog2e)), ex2(__fmul_rn(fabsf(v.y), -kLog2e)));
    const float2 s = __fadd2_rn(u, both(2.f));
    const float2 w = __fmul2_rn(u, make_float2(rcp_approx(s.x), rcp_approx(s.y))), q = __fmul2_rn(w, w);
    float2 p = __ffma2_rn(both(0.2817465662956238f), q, both(0.2796141803264618f));
    p = __ffma2_rn(p, q, both(0.40024852752685547f));
    p = __ffma2_rn(p, q, both(0.6666631698608398f));
    p = __ffma2_rn(p, q, both(2.f));
    return __ffma2_rn(p, w, m);
}
// Its derivative sigmoid(v), from the u that softplus2 left.
__device__ __forceinline__ float2 sigmoid2(const float2& v, const float2& u) {
    const float2 s = __fadd2_rn(u, both(1.f));
    const float a = rcp_approx(s.x), b = rcp_approx(s.y);
    return make_float2(v.x >= 0.f ? a : __fmul_rn(u.x, a), v.y >= 0.f ? b : __fmul_rn(u.y, b));
}
// silu(z) = z / (1 + e^-z) and, with it, sigmoid(z).
__device__ __forceinline__ float2 silu2(const float2& z, float2& sig) {
    const float2 e = __fmul2_rn(z, both(-kLog2e));
    const float2 s = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
    sig = make_float2(rcp_approx(s.x), rcp_approx(s.y));
    return __fmul2_rn(z, sig);
}

// The steps d of two (token, channel) pairs from the raw dt and the channels' biases.
__device__ __forceinline__ float2 step_of(const float2& raw, const float2& bias, bool use_softplus) {
    const float2 v = __fadd2_rn(raw, bias);
    float2 u;
    return use_softplus ? softplus2(v, u) : v;
}

// Two neighbouring states one token on: h <- exp2(d A2) h + dx B.
__device__ __forceinline__ void advance(float2& h, const float2& A2, const float2& d, const float2& dx,
                                        const float2& B) {
    const float2 e = __fmul2_rn(d, A2);
    h = __ffma2_rn(make_float2(ex2(e.x), ex2(e.y)), h, __fmul2_rn(dx, B));
}

struct Params {
    int N, T, C, G, CG, bpg;  // CG: channels per group, bpg: channel blocks per group
    int softplus;
    const void *x, *dt, *z, *B, *Cm;
    int64_t ldx, lddt, ldz, ldB, ldC;
    const float *A_log, *D, *bias;
    const int32_t* cu;
    float* state;
    const int32_t* idx;
    int num_slots;
    const int32_t* has_init;
    void* y;
    int ranked;  // prompts: take the sequences in order of length
};

__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four consecutive values as two packed pairs.
__device__ __forceinline__ void load4(const float* p, float2 (&v)[2]) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = make_float2(u.x, u.y), v[1] = make_float2(u.z, u.w);
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float2 (&v)[2]) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = make_float2(bf_lo(u.x), bf_hi(u.x)), v[1] = make_float2(bf_lo(u.y), bf_hi(u.y));
}

// Named barriers between a CTA's warps, and registers moved between its warpgroups.
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
template <int N> __device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_less() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Bounds of sequence n, whatever cu_seqlens holds.
__device__ __forceinline__ void bounds(const int32_t* cu, int n, int T, int& bos, int& eos) {
    bos = max(0, min(__ldg(cu + n), T));
    eos = max(bos, min(__ldg(cu + n + 1), T));
}

// Sum over a channel's states from the 4 a lane holds (L lanes per channel, lane j the states
// 4j .. 4j+3): the odd lane of a pair carries on its neighbour's chain.  Valid on odd lanes.
template <int L>
__device__ __forceinline__ float sum_states4(const float2 (&h)[2], const float2 (&c)[2], int j) {
    float2 p = __ffma2_rn(h[1], c[1], __fmul2_rn(h[0], c[0]));
    float2 q;
    q.x = __shfl_xor_sync(0xffffffffu, p.x, 1);
    q.y = __shfl_xor_sync(0xffffffffu, p.y, 1);
    if (j & 1) p = __ffma2_rn(h[1], c[1], __ffma2_rn(h[0], c[0], q));
    float s = __fadd_rn(p.x, p.y);
#pragma unroll
    for (int off = 2; off < L; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

}  // namespace scan

// Host side.

// Whether a kernel whose warpgroups move registers is launched with the `need` registers a CTA that
// they then hold: they would wait for ever for more.  GDN_ERR_UNSUPPORTED where it is not.  What the
// runtime answers holds for the process, an error of the runtime does not.
template <typename K>
gdn_status check_registers(K* kernel, int threads, int need, std::atomic<int>& known) {
    int ok = known.load(std::memory_order_relaxed);  // 0: not asked yet, 1: enough, -1: too few
    if (!ok) {
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess) return GDN_ERR_CUDA;
        ok = a.numRegs * threads < need ? -1 : 1;
        known.store(ok, std::memory_order_relaxed);
    }
    return ok > 0 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}
inline gdn_status check_scan(const gdn_scan_shape* s) {
    if (!s) return GDN_ERR_INVALID_ARG;
    if (s->N < 0 || s->T_total < 0 || s->C <= 0 || s->G <= 0 || s->C % s->G) return GDN_ERR_INVALID_ARG;
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (s->T_total > INT_MAX - 64) return GDN_ERR_UNSUPPORTED;
    if (s->S != 8 && s->S != 16 && s->S != 32 && s->S != 64) return GDN_ERR_UNSUPPORTED;
    if ((s->C / s->G) % 8) return GDN_ERR_UNSUPPORTED;
    if ((long long)s->N * s->C >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    const int64_t vn = s->dtype == GDN_BF16 ? 8 : 4;
    const int64_t bc = (int64_t)s->G * s->S;
    if (s->ldx < s->C || s->lddt < s->C || s->ldB < bc || s->ldC < bc) return GDN_ERR_INVALID_ARG;
    if (s->ldx % vn || s->lddt % vn || s->ldB % vn || s->ldC % vn) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace gdn
