// gdn_norm.cu -- RMSNorm with the residual's addition, in the same type or in 8 bits with scales, and
// its gradient.
//
//     s = round(x + residual),  r = (mean s^2 + eps)^-1/2,  y = s r w;   8 bits: scale = max |y| / 448 of a group, e4m3(y / scale)
//     g = d_y w:   dx = r (g - s r^2 mean(g s)) + d_residual_out,   dw = sum over rows of d_y s r
//
// Every value is read once and written once: HBM bounds it.  A row stays in the registers of a group of
// threads, lane i of it 16-byte chunks i, i + lanes, ..; a warp's sums are xor butterflies, a row's warps
// are added in ascending order.
#include <cuda_fp8.h>

#include "../../include/gdn_layer.h"
#include "gdn_host.h"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

struct NormParams {
    int64_t rows;
    int d, chunks, tpr;  // tpr: threads of a row
    int glanes;          // lanes of a group of values that share a scale (0: the row)
    int groups;          // scales of a row
    float c, eps;
    int64_t ldx, ldr;
    const void *x, *res, *dy, *dres;
    const float* w;
    void *res_out, *y;
    float *scales, *part;
};

struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return __fadd_rn(a, b); }
};
struct Max {
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// OP over the `lanes` (a power of two up to 32) neighbours of a lane.
template <typename OP>
__device__ __forceinline__ float over_lanes(float v, int lanes) {
    for (int off = 1; off < lanes; off <<= 1) v = OP::of(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
// OP over a row's threads.  Every thread of the CTA calls it; `buf` holds a value per warp.
template <typename OP>
__device__ __forceinline__ float over_row(float v, int tpr, float* buf) {
    v = over_lanes<OP>(v, tpr < 32 ? tpr : 32);
    if (tpr <= 32) return v;
    const int warp = threadIdx.x / 32, per = tpr / 32, first = warp / per * per;
    if (threadIdx.x % 32 == 0) buf[warp] = v;
    __syncthreads();
    v = buf[first];
    for (int i = 1; i < per; ++i) v = OP::of(v, buf[first + i]);
    __syncthreads();
    return v;
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void load_weight(const float* w, float (&v)[8]) {
    unpack(ld16(w), reinterpret_cast<float(&)[4]>(v[0]));
    unpack(ld16(w + 4), reinterpret_cast<float(&)[4]>(v[4]));
}
__device__ __forceinline__ void load_weight(const float* w, float (&v)[4]) { unpack(ld16(w), v); }

__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ void store_fp8(uint8_t* to, const float (&v)[8]) {
    *reinterpret_cast<uint2*>(to) = make_uint2(fp8x4(v[0], v[1], v[2], v[3]), fp8x4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store_fp8(uint8_t* to, const float (&v)[4]) { *reinterpret_cast<uint32_t*>(to) = fp8x4(v[0], v[1], v[2], v[3]); }

template <typename T, int NC, bool FP8>
__global__ void __launch_bounds__(1024) add_norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int VN = V16<T>::n;
    __shared__ float buf[32];
    const int lane = threadIdx.x % p.tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / p.tpr) + threadIdx.x / p.tpr;
    const bool live = row < p.rows;
    float v[NC][VN], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        if (live && c < p.chunks) {
            unpack(ld16_stream(static_cast<const T*>(p.x) + row * p.ldx + c * VN), v[i]);
            if (p.res) {
                float a[VN];
                unpack(ld16_stream(static_cast<const T*>(p.res) + row * p.ldr + c * VN), a);
#pragma unroll
                for (int e = 0; e < VN; ++e) v[i][e] = to_f(rounded<T>(__fadd_rn(v[i][e], a[e])));
            }
        } else {
#pragma unroll
            for (int e = 0; e < VN; ++e) v[i][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < VN; ++e) ss = __fmaf_rn(v[i][e], v[i][e], ss);
    }
    const float r = rsqrtf(__fmaf_rn(over_row<Sum>(ss, p.tpr, buf), p.c, p.eps));
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        const bool has = live && c < p.chunks;
        if (has && p.res) st16(static_cast<T*>(p.res_out) + row * p.d + c * VN, pack(v[i]));
        if (has) {
            float w[VN];
            load_weight(p.w + c * VN, w);
#pragma unroll
            for (int e = 0; e < VN; ++e) v[i][e] = __fmul_rn(__fmul_rn(v[i][e], r), w[e]);
        }
        if constexpr (!FP8) {
            if (has) st16(static_cast<T*>(p.y) + row * p.d + c * VN, pack(v[i]));
        } else {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < VN; ++e) m = fmaxf(m, fabsf(v[i][e]));
            if (p.glanes) {
                const float scale = fmaxf(__fmul_rn(over_lanes<Max>(m, p.glanes), 1.f / 448.f), 1.17549435e-38f), inv = __frcp_rn(scale);
#pragma unroll
                for (int e = 0; e < VN; ++e) v[i][e] = __fmul_rn(v[i][e], inv);
                if (has) store_fp8(static_cast<uint8_t*>(p.y) + row * p.d + c * VN, v[i]);
                if (has && lane % p.glanes == 0) p.scales[row * p.groups + c / p.glanes] = scale;
            } else {
                most = fmaxf(most, m);
            }
        }
    }
    if constexpr (FP8) {
        if (p.glanes) return;
        const float scale = fmaxf(__fmul_rn(over_row<Max>(most, p.tpr, buf), 1.f / 448.f), 1.17549435e-38f), inv = __frcp_rn(scale);
        if (live && lane == 0) p.scales[row] = scale;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (!live || c >= p.chunks) continue;
#pragma unroll
            for (int e = 0; e < VN; ++e) v[i][e] = __fmul_rn(v[i][e], inv);
            store_fp8(static_cast<uint8_t*>(p.y) + row * p.d + c * VN, v[i]);
        }
    }
}

template <typename T, int NC>
__global__ void __launch_bounds__(1024) add_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    constexpr int VN = V16<T>::n;
    __shared__ float buf[32];
    extern __shared__ float acc[];  // [rows of the CTA][d]
    const int lane = threadIdx.x % p.tpr, per = blockDim.x / p.tpr, mine = threadIdx.x / p.tpr;
    float dw[NC][VN];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < VN; ++e) dw[i][e] = 0.f;
    for (int64_t first = (int64_t)blockIdx.x * per; first < p.rows; first += (int64_t)gridDim.x * per) {
        const int64_t row = first + mine;
        const bool live = row < p.rows;
        float v[NC][VN], g[NC][VN], ss = 0.f, gx = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (live && c < p.chunks) {
                unpack(ld16_stream(static_cast<const T*>(p.x) + row * p.ldx + c * VN), v[i]);
                unpack(ld16_stream(static_cast<const T*>(p.dy) + row * p.d + c * VN), g[i]);
            } else {
#pragma unroll
                for (int e = 0; e < VN; ++e) v[i][e] = g[i][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VN; ++e) ss = __fmaf_rn(v[i][e], v[i][e], ss);
        }
        const float r = rsqrtf(__fmaf_rn(over_row<Sum>(ss, p.tpr, buf), p.c, p.eps));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (!live || c >= p.chunks) continue;
            float w[VN];
            load_weight(p.w + c * VN, w);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                dw[i][e] = __fmaf_rn(__fmul_rn(v[i][e], r), g[i][e], dw[i][e]);
                g[i][e] = __fmul_rn(g[i][e], w[e]);
                gx = __fmaf_rn(g[i][e], v[i][e], gx);
            }
        }
        // r (g - s (r sum(g s)) (r c)): these products stay in range where r^3 is not
        const float f = -__fmul_rn(__fmul_rn(r, over_row<Sum>(gx, p.tpr, buf)), __fmul_rn(r, p.c));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            if (!live || c >= p.chunks) continue;
            float o[VN];
            if (p.dres) unpack(ld16_stream(static_cast<const T*>(p.dres) + row * p.d + c * VN), o);
#pragma unroll
            for (int e = 0; e < VN; ++e) o[e] = __fmaf_rn(r, __fmaf_rn(v[i][e], f, g[i][e]), p.dres ? o[e] : 0.f);
            st16(static_cast<T*>(p.y) + row * p.d + c * VN, pack(o));
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = lane + i * p.tpr;
        if (c >= p.chunks) continue;
#pragma unroll
        for (int e = 0; e < VN; ++e) acc[(int64_t)mine * p.d + c * VN + e] = dw[i][e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.d; e += blockDim.x) {
        float s = acc[e];
        for (int i = 1; i < per; ++i) s = __fadd_rn(s, acc[(int64_t)i * p.d + e]);
        p.part[(int64_t)blockIdx.x * p.d + e] = s;
    }
}

// dweight: the CTAs' partials.  A CTA takes 4 float4 columns; thread (slice, column) adds partials slice,
// slice + 64, .., then a thread per column the slices in order.
__global__ void __launch_bounds__(256) add_norm_sum_kernel(int d, int ctas, const float* __restrict__ part, float* __restrict__ out) {
    __shared__ float4 sums[64][4];
    const int x = threadIdx.x & 3, slice = threadIdx.x >> 2, e = (blockIdx.x * 4 + x) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v) { s.x = __fadd_rn(s.x, v.x), s.y = __fadd_rn(s.y, v.y), s.z = __fadd_rn(s.z, v.z), s.w = __fadd_rn(s.w, v.w); };
    if (e < d) {
#pragma unroll 4
        for (int i = slice; i < ctas; i += 64) add(*reinterpret_cast<const float4*>(part + (int64_t)i * d + e));
    }
    sums[slice][x] = s;
    __syncthreads();
    if (slice || e >= d) return;
    for (int i = 1; i < 64; ++i) add(sums[i][x]);
    *reinterpret_cast<float4*>(out + e) = s;
}

constexpr int kMaxWidth = 16384, kMaxChunks = 4;  // chunks a thread holds

gdn_status check_norm(const gdn_add_norm_shape* s) {
    if (!s) return GDN_ERR_INVALID_ARG;
    if (s->rows < 0 || s->d <= 0) return GDN_ERR_INVALID_ARG;
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    const int vn = s->dtype == GDN_BF16 ? 8 : 4;
    if (s->d % vn || s->d > kMaxWidth || s->rows >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    if (!(s->eps >= 0.f) || s->ldx < s->d || s->ldx % vn) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Threads of a row: one chunk each up to a warp, then up to kMaxChunks.
NormParams norm_params(const gdn_add_norm_shape* s) {
    NormParams p{};
    p.rows = s->rows, p.d = s->d, p.eps = s->eps, p.c = 1.f / (float)s->d, p.ldx = s->ldx, p.ldr = s->ldr;
    p.chunks = s->d / (s->dtype == GDN_BF16 ? 8 : 4);
    p.tpr = 1;
    while (p.tpr < p.chunks && (p.tpr < 32 || p.tpr * kMaxChunks < p.chunks)) p.tpr *= 2;
    return p;
}
int cta_threads(const NormParams& p) { return p.tpr > 256 ? p.tpr : 256; }
int bwd_ctas(const NormParams& p) {
    const int threads = cta_threads(p);
    const int64_t want = (p.rows * p.tpr + threads - 1) / threads, most = (int64_t)kSMs * (threads > 512 ? 1 : 2);
    return (int)(want < most ? (want > 1 ? want : 1) : most);
}

// K<T, NC>::go(grid, threads, stream, p)
template <template <typename, int> class K, typename T>
gdn_status by_chunks(int grid, cudaStream_t s, const NormParams& p) {
    const int nc = (p.chunks + p.tpr - 1) / p.tpr, threads = cta_threads(p);
    if (nc <= 1) return K<T, 1>::go(grid, threads, s, p);
    if (nc == 2) return K<T, 2>::go(grid, threads, s, p);
    return K<T, 4>::go(grid, threads, s, p);
}
template <typename T, int NC>
struct SameK {
    static gdn_status go(int grid, int threads, cudaStream_t s, const NormParams& p) {
        add_norm_kernel<T, NC, false><<<grid, threads, 0, s>>>(p);
        return launch_status();
    }
};
template <typename T, int NC>
struct Fp8K {
    static gdn_status go(int grid, int threads, cudaStream_t s, const NormParams& p) {
        add_norm_kernel<T, NC, true><<<grid, threads, 0, s>>>(p);
        return launch_status();
    }
};
template <typename T, int NC>
struct BwdK {
    static gdn_status go(int grid, int threads, cudaStream_t s, const NormParams& p) {
        const size_t smem = p.part ? (size_t)(threads / p.tpr) * p.d * sizeof(float) : 0;
        if (smem > 48 * 1024 - 256 && cudaFuncSetAttribute(add_norm_bwd_kernel<T, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return GDN_ERR_CUDA;
        add_norm_bwd_kernel<T, NC><<<grid, threads, smem, s>>>(p);
        return launch_status();
    }
};

gdn_status norm_fwd(const gdn_add_norm_shape* shape, const void* x, const void* res, const float* w, void* res_out, void* y,
                    float* scales, bool fp8, void* stream) {
    gdn_status st = check_norm(shape);
    if (st != GDN_OK) return st;
    const int vn = shape->dtype == GDN_BF16 ? 8 : 4;
    if (fp8 && shape->group != 0 && shape->group != 32 && shape->group != 64 && shape->group != 128) return GDN_ERR_UNSUPPORTED;
    if (shape->rows == 0) return GDN_OK;
    if (!x || !w || !y || (res && !res_out) || (fp8 && !scales)) return GDN_ERR_INVALID_ARG;
    if (res && (shape->ldr < shape->d || shape->ldr % vn)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(res) || !aligned16(w) || !aligned16(res_out) || !aligned16(y) || !aligned4(scales)) return GDN_ERR_INVALID_ARG;
    const void* to[] = {y, res ? res_out : nullptr};
    for (int i = fp8 ? 1 : 0; i < 2; ++i)
        if (to[i] && ((to[i] == x && shape->ldx != shape->d) || (to[i] == res && shape->ldr != shape->d))) return GDN_ERR_INVALID_ARG;
    if ((to[1] && y == to[1]) || (fp8 && (y == x || y == res || scales == y || scales == x || scales == res || scales == to[1]))) return GDN_ERR_INVALID_ARG;
    NormParams p = norm_params(shape);
    p.x = x, p.res = res, p.w = w, p.res_out = res_out, p.y = y, p.scales = scales;
    // A group that takes in the whole row is the row.
    const int lanes = shape->group / vn;
    p.glanes = lanes >= p.chunks ? 0 : lanes, p.groups = p.glanes ? (p.chunks + lanes - 1) / lanes : 1;
    const int rows = cta_threads(p) / p.tpr;
    const int grid = (int)((p.rows + rows - 1) / rows);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (shape->dtype == GDN_BF16) return fp8 ? by_chunks<Fp8K, __nv_bfloat16>(grid, s, p) : by_chunks<SameK, __nv_bfloat16>(grid, s, p);
    return fp8 ? by_chunks<Fp8K, float>(grid, s, p) : by_chunks<SameK, float>(grid, s, p);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_add_rmsnorm(const gdn_add_norm_shape* shape, const void* x, const void* residual, const float* weight,
                                      void* residual_out, void* y, void* stream) {
    return gdn::norm_fwd(shape, x, residual, weight, residual_out, y, nullptr, false, stream);
}

extern "C" gdn_status gdn_add_rmsnorm_fp8(const gdn_add_norm_shape* shape, const void* x, const void* residual, const float* weight,
                                          void* residual_out, void* y, float* scales, void* stream) {
    return gdn::norm_fwd(shape, x, residual, weight, residual_out, y, scales, true, stream);
}

extern "C" size_t gdn_add_rmsnorm_bwd_workspace_size(const gdn_add_norm_shape* shape) {
    using namespace gdn;
    if (check_norm(shape) != GDN_OK) return 0;
    return (size_t)bwd_ctas(norm_params(shape)) * shape->d * sizeof(float);
}

extern "C" gdn_status gdn_add_rmsnorm_bwd(const gdn_add_norm_shape* shape, const void* s, const float* weight, const void* d_y,
                                          const void* d_residual_out, void* dx, float* dweight, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    using namespace gdn;
    gdn_status st = check_norm(shape);
    if (st != GDN_OK) return st;
    const bool rows = shape->rows > 0;
    if (rows && (!s || !weight || !d_y || !dx)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(s) || !aligned16(weight) || !aligned16(d_y) || !aligned16(d_residual_out) || !aligned16(dx) || !aligned16(dweight)) return GDN_ERR_INVALID_ARG;
    if (rows && dx == s && shape->ldx != shape->d) return GDN_ERR_INVALID_ARG;
    if (dweight && (!workspace || !aligned16(workspace) || workspace_bytes < gdn_add_rmsnorm_bwd_workspace_size(shape))) return GDN_ERR_WORKSPACE;
    if (!rows && !dweight) return GDN_OK;
    NormParams p = norm_params(shape);
    p.x = s, p.w = weight, p.dy = d_y, p.dres = d_residual_out, p.y = dx, p.part = dweight ? static_cast<float*>(workspace) : nullptr;
    const int ctas = bwd_ctas(p);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = shape->dtype == GDN_BF16 ? by_chunks<BwdK, __nv_bfloat16>(ctas, cs, p) : by_chunks<BwdK, float>(ctas, cs, p);
    if (st != GDN_OK || !dweight) return st;
    add_norm_sum_kernel<<<(unsigned)((p.d + 15) / 16), 256, 0, cs>>>(p.d, ctas, p.part, dweight);
    return launch_status();
}
