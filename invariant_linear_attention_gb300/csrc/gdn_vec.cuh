// gdn_vec.cuh -- what the streaming layer kernels share: 16-byte vectors of bf16 or fp32
// values, and SiLU with the hardware exponential.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

constexpr int kSMs = 152;

// ---------------------------------------------------------------- 16-byte vectors
template <typename T>
struct V16;
template <>
struct V16<float> {
    static constexpr int n = 4;
};
template <>
struct V16<__nv_bfloat16> {
    static constexpr int n = 8;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
    f[0] = bf_lo(u.x), f[1] = bf_hi(u.x), f[2] = bf_lo(u.y), f[3] = bf_hi(u.y);
    f[4] = bf_lo(u.z), f[5] = bf_hi(u.z), f[6] = bf_lo(u.w), f[7] = bf_hi(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z),
    f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(bf_pack(f[0], f[1]), bf_pack(f[2], f[3]), bf_pack(f[4], f[5]), bf_pack(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}

__device__ __forceinline__ uint4 ld16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint4 ld16_stream(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void st16(void* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }
__device__ __forceinline__ void st16_stream(void* p, const uint4& v) { __stcs(reinterpret_cast<uint4*>(p), v); }

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// SiLU on the streaming paths (conv output, RMSNorm gate): x * (1 / (1 + e^-x))
// with the hardware exponential and the hardware approximate reciprocal, a
// few ulp (far below the bf16 rounding of the outputs) at a fraction of the
// instruction count, which these HBM-bound kernels would otherwise be limited
// by.  The reciprocal is the bare rcp.approx.ftz instruction: for x < -87 the
// exponential overflows to +inf and 1 / inf = 0, the limit SiLU has there.
// Deterministic, and one function for every kernel, so prefill and decode
// agree bit for bit.
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float silu_fast(float x) { return __fmul_rn(x, rcp_approx(__fadd_rn(1.f, __expf(-x)))); }

// 2^x by the bare hardware exponential: __expf also rescales around subnormal results, four more
// instructions that 1 + e^x does not need.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace gdn
