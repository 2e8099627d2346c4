// gdn_norm.cu -- RMSNorm with the residual's addition, in the same type or in 8 bits with scales, and
// its gradient.
//
//     s = round(x + residual),  r = (mean s^2 + eps)^-1/2,  y = s r w;   8 bits: scale = max |y| / 448 of a group, e4m3(y / scale)
//     g = d_y w:   dx = r (g - s r^2 mean(g s)) + d_residual_out,   dw = sum over rows of d_y s r
//
// Every value is read once and written once: HBM bounds it.  A row stays in the registers of a group of
// threads, lane i of it 16-byte chunks i, i + lanes, ..; sums are xor butterflies, in the warps and then over a row's warps.
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
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
        if (off < lanes) v = OP::of(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
// OP over a row's threads, of N values at once: in the warps, then over the warps' results.  Every thread of the CTA
// calls it; `buf` holds N values per warp, and the next call has another one.
template <typename OP, int N>
__device__ __forceinline__ void over_row(float (&v)[N], int tpr, float (&buf)[N][32]) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = over_lanes<OP>(v[k], tpr < 32 ? tpr : 32);
    if (tpr <= 32) return;
    const int warp = threadIdx.x / 32, per = tpr / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) buf[k][warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = over_lanes<OP>(buf[k][(warp & -per) + (lane & (per - 1))], per);
}

__device__ __forceinline__ void load_weight(const float* w, float (&v)[8]) {
    unpack(ld16(w), reinterpret_cast<float(&)[4]>(v[0]));
    unpack(ld16(w + 4), reinterpret_cast<float(&)[4]>(v[4]));
}
__device__ __forceinline__ void load_weight(const float* w, float (&v)[4]) { unpack(ld16(w), v); }

__device__ __forceinline__ uint32_t fp8x4(const float2& a, const float2& b) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3), hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ void store_fp8(uint8_t* to, const float2 (&v)[4]) { *reinterpret_cast<uint2*>(to) = make_uint2(fp8x4(v[0], v[1]), fp8x4(v[2], v[3])); }
__device__ __forceinline__ void store_fp8(uint8_t* to, const float2 (&v)[2]) { *reinterpret_cast<uint32_t*>(to) = fp8x4(v[0], v[1]); }

constexpr float kTop = 448.f, kLeast = 1.17549435e-38f;  // e4m3's largest value; the smallest scale, 2^-126

// A group's scale and the factor that takes its values t = s w to 8 bits.  The scale is the norm's r max|t| / 448, but the
// values go by 448 / max|t|: r's error and a rounding each stay out of them.  The reciprocal is the hardware's with
// a step of Newton's method.  (Where that is past fp32, in a group of next to nothing, and where the scale is the smallest one and
// not the group's, the values are multiplied by r and go by the scale.)
struct Scale {
    float scale, by;
    bool tiny;
    template <int NP>
    __device__ __forceinline__ void apply(float2 (&v)[NP], float r) const {
        if (tiny) {
#pragma unroll
            for (int e = 0; e < NP; ++e) v[e] = __fmul2_rn(v[e], make_float2(r, r));
        }
#pragma unroll
        for (int e = 0; e < NP; ++e) v[e] = __fmul2_rn(v[e], make_float2(by, by));
    }
};
__device__ __forceinline__ Scale scale_of(float most, float r) {
    Scale s;
    const float own = __fmul_rn(__fmul_rn(most, r), 1.f / kTop);
    s.scale = fmaxf(own, kLeast);
    s.tiny = !(most > 1e-30f && own > kLeast);
    const float x = s.tiny ? s.scale : most, y = rcp_approx(x);
    const float z = __fmaf_rn(y, __fmaf_rn(-x, y, 1.f), y);
    s.by = __fmaf_rn(r, 0.f, s.tiny ? y : __fmul_rn(kTop, most < 1e38f ? z : y));  // a row whose r is not a number has no values
    return s;
}

__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

// A CTA takes rows blockIdx.x, + gridDim.x, ..  Up to two chunks a thread (NC), it keeps its weights in registers and
// has the next row's loads under way while a row is summed and stored.  A row waits packed, as it is stored.  Its places
// in memory are pointers that go on by a fixed step (addresses from the row's number: 174 us for the 8-bit case below, so 157; its
// reductions unrolled 149).
//
// HBM bounds it: 32768 x 4096, bf16, residual: 161 us, 0.98 of the measured peak; in 8 bits with a scale for each 128 values 149 us,
// 0.93, with 69 % of the issue slots taken.  Without a residual the 8-bit form has half the bytes for the same instructions
// and is bound by them (120 us, 0.50).
template <typename T, int NC, int NT, bool FP8>
__global__ void __launch_bounds__(NT, NT <= 256 ? 3 : NT == 512 && NC <= 2 ? 2 : 1) add_norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int VN = V16<T>::n, NP = VN / 2;
    constexpr bool ahead = NC <= 2, early = NT < 1024;  // the registers of 1024 threads hold one row
    __shared__ float buf[2][1][32], buf2[2][1][32];
    const int lane = threadIdx.x % p.tpr, per = NT / p.tpr;
    const bool res = p.res != nullptr;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const int64_t step = (int64_t)gridDim.x * per;
    int64_t first = (int64_t)blockIdx.x * per, row = first + threadIdx.x / p.tpr;
    const int far = p.tpr * VN;  // from one of a thread's chunks to the next
    bool in[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) in[i] = lane + i * p.tpr < p.chunks;
    const T* px = static_cast<const T*>(p.x) + row * p.ldx + lane * VN;
    const T* pr = res ? static_cast<const T*>(p.res) + row * p.ldr + lane * VN : nullptr;
    T* po = res ? static_cast<T*>(p.res_out) + row * p.d + lane * VN : nullptr;
    T* py = static_cast<T*>(p.y) + (FP8 ? 0 : row * p.d + lane * VN);
    uint8_t* pq = static_cast<uint8_t*>(p.y) + (FP8 ? row * p.d + lane * VN : 0);
    const int64_t sx = step * p.ldx, sr = step * p.ldr, sd = step * p.d;
    uint4 a[NC], b[NC];
    auto load = [&](bool live) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            a[i] = live && in[i] ? ld16_stream(px + i * far) : none;
            b[i] = live && in[i] && res ? ld16_stream(pr + i * far) : none;
        }
    };
    float2 wk[ahead ? NC : 1][NP];
    auto weight = [&](int i, float2 (&w)[NP]) {
        if (!in[i]) return;
#pragma unroll
        for (int e = 0; e < NP; e += 2) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p.w + (lane + i * p.tpr) * VN + 2 * e));
            w[e] = make_float2(v.x, v.y), w[e + 1] = make_float2(v.z, v.w);
        }
    };
    auto values = [&](int i, const uint4& s, float2 (&v)[NP]) {  // s w
        unpack2(s, v);
        if constexpr (!ahead) weight(i, wk[0]);
#pragma unroll
        for (int e = 0; e < NP; ++e) v[e] = __fmul2_rn(v[e], wk[ahead ? i : 0][e]);
    };
    auto largest = [&](const float2 (&v)[NP]) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < NP; ++e) m = fmaxf(m, fmaxf(fabsf(v[e].x), fabsf(v[e].y)));
        return m;
    };
    if constexpr (ahead) {
#pragma unroll
        for (int i = 0; i < NC; ++i) weight(i, wk[i]);
    }
    if (early) load(row < p.rows);
    for (int turn = 0; first < p.rows; first += step, turn ^= 1) {
        const bool live = row < p.rows;
        if (!early) load(live);
        uint4 s[NC];
        float2 s2 = twice(0.f);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float2 v[NP];
            s[i] = a[i];
            unpack2(a[i], v);
            if (res) {
                float2 add[NP];
                unpack2(b[i], add);
#pragma unroll
                for (int e = 0; e < NP; ++e) v[e] = __fadd2_rn(v[e], add[e]);
                s[i] = pack2(v);
                unpack2(s[i], v);
                if (live && in[i]) st16_stream(po + i * far, s[i]);
            }
#pragma unroll
            for (int e = 0; e < NP; ++e) s2 = __ffma2_rn(v[e], v[e], s2);
        }
        px += sx, pr += sr, po += sd;
        if (early) load(row + step < p.rows);
        float ss[1] = {__fadd_rn(s2.x, s2.y)};
        over_row<Sum>(ss, p.tpr, buf[turn]);
        const float r = rsqrtf(__fmaf_rn(ss[0], p.c, p.eps));
        if constexpr (!FP8) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float2 v[NP];
                unpack2(s[i], v);
                if constexpr (!ahead) weight(i, wk[0]);
#pragma unroll
                for (int e = 0; e < NP; ++e) v[e] = __fmul2_rn(__fmul2_rn(v[e], twice(r)), wk[ahead ? i : 0][e]);
                if (live && in[i]) st16_stream(py + i * far, pack2(v));
            }
            py += sd;
        } else if (p.glanes) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float2 v[NP];
                values(i, s[i], v);
                const Scale sc = scale_of(over_lanes<Max>(in[i] ? largest(v) : 0.f, p.glanes), r);
                sc.apply(v, r);
                if (live && in[i]) {
                    store_fp8(pq + i * far, v);
                    if (lane % p.glanes == 0) p.scales[row * p.groups + (lane + i * p.tpr) / p.glanes] = sc.scale;
                }
            }
            pq += sd;
        } else {
            float most[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float2 v[NP];
                if (!in[i]) continue;
                values(i, s[i], v);
                most[0] = fmaxf(most[0], largest(v));
            }
            over_row<Max>(most, p.tpr, buf2[turn]);
            const Scale sc = scale_of(most[0], r);
            if (live && lane == 0) p.scales[row] = sc.scale;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float2 v[NP];
                values(i, s[i], v);
                sc.apply(v, r);
                if (live && in[i]) store_fp8(pq + i * far, v);
            }
            pq += sd;
        }
        row += step;
    }
}

// The gradient takes rows the same way.  sum(g s) needs no r, so that both sums go together.  dw: a thread's
// columns in registers, with more than two chunks in its own places of shared memory.  32768 x 4096, bf16, with the residual's
// gradient: 171 us, 0.93 of HBM; rows past 8192 (fp32 4096) values hold more than the registers do: 8192 x 16384 277 us, 0.57.
template <typename T, int NC, int NT>
__global__ void __launch_bounds__(NT, NT <= 256 ? 2 : 1) add_norm_bwd_kernel(const __grid_constant__ NormParams p) {
    constexpr int VN = V16<T>::n;
    constexpr bool ahead = NC <= 2;
    __shared__ float buf[2][2][32];
    extern __shared__ __align__(16) float acc[];  // [rows of the CTA][d]
    const int lane = threadIdx.x % p.tpr, per = NT / p.tpr, mine = threadIdx.x / p.tpr;
    const bool res = p.dres != nullptr;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 xn[NC], gn[NC], rn[NC];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = lane + i * p.tpr;
            const bool has = row < p.rows && c < p.chunks;
            xn[i] = has ? ld16_stream(static_cast<const T*>(p.x) + row * p.ldx + c * VN) : none;
            gn[i] = has ? ld16_stream(static_cast<const T*>(p.dy) + row * p.d + c * VN) : none;
            rn[i] = has && res ? ld16_stream(static_cast<const T*>(p.dres) + row * p.d + c * VN) : none;
        }
    };
    float wk[ahead ? NC : 1][VN], dw[ahead ? NC : 1][VN];
    auto weight = [&](int i, float (&w)[VN]) {
        if (lane + i * p.tpr < p.chunks) load_weight(p.w + (lane + i * p.tpr) * VN, w);
    };
    auto put = [&](int i, const float (&v)[VN]) {
        float4* to = reinterpret_cast<float4*>(acc + (int64_t)mine * p.d + (lane + i * p.tpr) * VN);
#pragma unroll
        for (int e = 0; e < VN; e += 4) to[e / 4] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float (&d)[VN] = dw[ahead ? i : 0], (&w)[VN] = wk[ahead ? i : 0];
#pragma unroll
        for (int e = 0; e < VN; ++e) w[e] = d[e] = 0.f;
        if constexpr (ahead) weight(i, w);
        else if (p.part && lane + i * p.tpr < p.chunks) put(i, d);
    }
    const int64_t step = (int64_t)gridDim.x * per;
    int64_t first = (int64_t)blockIdx.x * per;
    load(first + mine);
    for (int turn = 0; first < p.rows; first += step, turn ^= 1) {
        const int64_t row = first + mine;
        uint4 xs[NC], gs[NC], rs[NC];
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float v[VN], g[VN];
            xs[i] = xn[i], gs[i] = gn[i], rs[i] = rn[i];
            unpack(xs[i], v);
            unpack(gs[i], g);
            if constexpr (!ahead) weight(i, wk[0]);
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                sums[0] = __fmaf_rn(v[e], v[e], sums[0]);
                sums[1] = __fmaf_rn(__fmul_rn(g[e], wk[ahead ? i : 0][e]), v[e], sums[1]);
            }
        }
        if constexpr (ahead) load(row + step);
        over_row<Sum>(sums, p.tpr, buf[turn]);
        const float r = rsqrtf(__fmaf_rn(sums[0], p.c, p.eps));
        // r (g - s (r sum(g s)) (r c)): these products stay in range where r^3 is not
        const float f = -__fmul_rn(__fmul_rn(r, sums[1]), __fmul_rn(r, p.c));
        if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = lane + i * p.tpr;
                if (c >= p.chunks) continue;
                float v[VN], g[VN], o[VN];
                unpack(xs[i], v);
                unpack(gs[i], g);
                unpack(rs[i], o);
                float (&d)[VN] = dw[ahead ? i : 0];
                if constexpr (!ahead) {
                    weight(i, wk[0]);
                    if (p.part) {
#pragma unroll
                        for (int e = 0; e < VN; e += 4) unpack(*reinterpret_cast<const uint4*>(acc + (int64_t)mine * p.d + c * VN + e), reinterpret_cast<float(&)[4]>(d[e]));
                    }
                }
#pragma unroll
                for (int e = 0; e < VN; ++e) {
                    d[e] = __fmaf_rn(__fmul_rn(v[e], r), g[e], d[e]);
                    o[e] = __fmaf_rn(r, __fmaf_rn(v[e], f, __fmul_rn(g[e], wk[ahead ? i : 0][e])), o[e]);
                }
                st16_stream(static_cast<T*>(p.y) + row * p.d + c * VN, pack(o));
                if constexpr (!ahead) {
                    if (p.part) put(i, d);
                }
            }
        }
        if constexpr (!ahead) load(row + step);
    }
    if (!p.part) return;
    if constexpr (ahead) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (lane + i * p.tpr < p.chunks) put(i, dw[i]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.d; e += NT) {
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

constexpr int kRowThreads = 256;  // of a CTA, unless a row has more
constexpr int kMaxWidth = 16384;

gdn_status check_norm(const gdn_add_norm_shape* s) {
    if (!s) return GDN_ERR_INVALID_ARG;
    if (s->rows < 0 || s->d <= 0) return GDN_ERR_INVALID_ARG;
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    const int vn = s->dtype == GDN_BF16 ? 8 : 4;
    if (s->d % vn || s->d > kMaxWidth || s->rows >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    if (!(s->eps >= 0.f) || s->ldx < s->d || s->ldx % vn) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// Threads of a row: one chunk each up to a warp, then up to two, from 512 threads on up to four.
NormParams norm_params(const gdn_add_norm_shape* s) {
    NormParams p{};
    p.rows = s->rows, p.d = s->d, p.eps = s->eps, p.c = 1.f / (float)s->d, p.ldx = s->ldx, p.ldr = s->ldr;
    p.chunks = s->d / (s->dtype == GDN_BF16 ? 8 : 4);
    p.tpr = 1;
    while (p.tpr < p.chunks && (p.tpr < 32 || p.tpr * (p.tpr < 512 ? 2 : 4) < p.chunks)) p.tpr *= 2;
    return p;
}
int cta_threads(const NormParams& p) { return p.tpr > kRowThreads ? p.tpr : kRowThreads; }
// CTAs that walk the rows: `each` threads an SM, a row for every group of threads at least.
int ctas_for(const NormParams& p, int each) {
    const int threads = cta_threads(p);
    const int64_t per = threads / p.tpr, want = (p.rows + per - 1) / per, most = (int64_t)kSMs * (each > threads ? each / threads : 1);
    return (int)(want < most ? (want > 1 ? want : 1) : most);
}
int bwd_ctas(const NormParams& p) { return ctas_for(p, 512); }

// K<T, NC, NT>::go(grid, stream, p)
template <template <typename, int, int> class K, typename T>
gdn_status by_chunks(int grid, cudaStream_t s, const NormParams& p) {
    const int nc = (p.chunks + p.tpr - 1) / p.tpr;
    if (nc <= 1) return K<T, 1, kRowThreads>::go(grid, s, p);
    if (nc == 2) return p.tpr <= kRowThreads ? K<T, 2, kRowThreads>::go(grid, s, p) : K<T, 2, 512>::go(grid, s, p);
    if constexpr (sizeof(T) == 4) {
        if (p.tpr > 512) return K<T, 4, 1024>::go(grid, s, p);
    }
    return K<T, 4, 512>::go(grid, s, p);
}
template <typename T, int NC, int NT>
struct SameK {
    static gdn_status go(int grid, cudaStream_t s, const NormParams& p) {
        add_norm_kernel<T, NC, NT, false><<<grid, NT, 0, s>>>(p);
        return launch_status();
    }
};
template <typename T, int NC, int NT>
struct Fp8K {
    static gdn_status go(int grid, cudaStream_t s, const NormParams& p) {
        add_norm_kernel<T, NC, NT, true><<<grid, NT, 0, s>>>(p);
        return launch_status();
    }
};
template <typename T, int NC, int NT>
struct BwdK {
    static gdn_status go(int grid, cudaStream_t s, const NormParams& p) {
        const size_t smem = p.part ? (size_t)(NT / p.tpr) * p.d * sizeof(float) : 0;
        if (smem > 47 * 1024 && cudaFuncSetAttribute(add_norm_bwd_kernel<T, NC, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return GDN_ERR_CUDA;
        add_norm_bwd_kernel<T, NC, NT><<<grid, NT, smem, s>>>(p);
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
    if (!aligned16(x) || !aligned16(res) || !aligned16(w) || !aligned16(res_out) || !aligned4(scales)) return GDN_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(y) & (fp8 ? 7u : 15u)) return GDN_ERR_INVALID_ARG;  // 8 bits: a chunk's values are one store of 8 or 4 bytes
    const void* to[] = {y, res ? res_out : nullptr};
    for (int i = fp8 ? 1 : 0; i < 2; ++i)
        if (to[i] && ((to[i] == x && shape->ldx != shape->d) || (to[i] == res && shape->ldr != shape->d))) return GDN_ERR_INVALID_ARG;
    if ((to[1] && y == to[1]) || (fp8 && (y == x || y == res || scales == y || scales == x || scales == res || scales == to[1]))) return GDN_ERR_INVALID_ARG;
    NormParams p = norm_params(shape);
    p.x = x, p.res = res, p.w = w, p.res_out = res_out, p.y = y, p.scales = scales;
    // A group that takes in the whole row is the row.
    const int lanes = shape->group / vn;
    p.glanes = lanes >= p.chunks ? 0 : lanes, p.groups = p.glanes ? (p.chunks + lanes - 1) / lanes : 1;
    const int grid = ctas_for(p, p.tpr > kRowThreads ? 1024 : 12 * kRowThreads);
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
    if (rows && (!s || !d_y || !dx)) return GDN_ERR_INVALID_ARG;
    if ((rows || dweight) && !weight) return GDN_ERR_INVALID_ARG;  // without rows dweight is written by the same kernels, which read the weight
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
