// gdn_scan_bwd.cu -- gradient of the selective scan.  With e = d_y silu(z), g the gradient with
// respect to h and G = a g what of it reaches the token before:
//
//     g_t = e_t C_t + G_{t+1}               (G = d_final_state behind the last token)
//     dC = sum_c e h,  dB = sum_c g d x,  u = sum_s g B,  w = G_t h_{t-1}
//     dx = d u + D e,  dd = x u + sum_s w A,  ddt = dd softplus',  dz = d_y (y / silu) silu'
//     dA_log = A sum_t w d,  dD = sum_t e x,  ddt_bias = sum_t ddt,  d_init_state = G_0
//
// A training batch has few sequences, and a walk is bound by its own latency, so the sequences
// are cut into segments of m tiles of 8 tokens that are walked side by side:
//   1. local: every segment's final state from a zero start, its G from a zero end (both in one
//      forward pass, with the running product of the decays), the states at its tiles' starts
//      and the sums of d up to there;
//   2. join: along each sequence, the segments' true start states and end G's;
//   3. grad: per segment, tiles last to first.  A tile's states are recomputed from its start into
//      registers, and its tokens walked backwards, on four warps; softplus and the gates before
//      and dx, ddt, dz and the sums of dB and dC after are other warps' work;
//   4. sums: the channel blocks' partials of dB and dC, the segments' of the parameters' gradients.
// Every sum's order is fixed by the shapes and cu_seqlens.
//
// The fp32 pipe and the instruction issue bound 1 and 3: per state and token 6 products or sums
// (packed by twos) and 1 exponential in 1, 13 and 2 in 3; HBM traffic is 11 (T, C) tensors (x, dt, d_y and z
// read by both, dx, ddt and dz written; 8 without a gate), 4 S bytes per channel and tile for the tiles'
// states, written and read once, and the segments' states.
#include "gdn_async.cuh"
#include "gdn_host.h"
#include "gdn_scan.cuh"

namespace gdn {
namespace {

using namespace scan;

constexpr int kTile = 8;
constexpr float kLn2 = 0.6931471805599453f;

struct BwdParams {
    Params f;
    int m;  // tiles per segment
    const float *h0, *dhT;
    const void* dy;
    void *dx, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *dbias, *dh0;
    // Workspace.  Segment k of sequence n is number cu[n] / (m kTile) + n + k (never two on one): as many
    // as the sequences have segments, but no fewer than one each.  A tile that is not its sequence's first
    // has the number t0 / kTile - 1 of its first token t0: T / kTile numbers, never two on one, for the last such
    // tile of a sequence starts before its end and the first of the next one kTile behind it.
    float* tiles;  // [T / kTile, C, S] the state at the tile's start, from a zero start of its segment (not of a segment's first)
    float* cum;    // [T / kTile, C] sum of d up to the tile's start
    float* seg_h;  // [segments, C, S] local final state, then the true start state
    float* seg_g;  // [segments, C, S] local G, then the true end G, then the segment's part of dA
    float* seg_d;  // [segments, C] sum of d
    float* bc;     // [channel blocks, T, 2, S] parts of dB and dC
    float *pD, *pb;  // [segments, C]
};

// Channels and threads of a CTA: a lane holds 4 states (L = S / 4 lanes a channel) of Q channels.
__host__ __device__ constexpr int channels_of(int S) { return S <= 16 ? 64 : 32; }
template <typename T, int S, int Q>
struct Geo {
    static constexpr int L = S / 4, CB = channels_of(S), NT = CB * L / Q;
    static_assert(NT % 32 == 0, "whole warps");
};

// Both walks read {d, d x, e, softplus'} per (token, channel), and B and C in fp32, from shared memory.
// Channel c of a token lies at float4 place(c): threads that write 8 (or 4) neighbours and lanes
// that read one each all miss each other's banks.  Zeros where there is no token or no channel:
// such a step has a = 1 and adds nothing.
__device__ __forceinline__ int place(int c) { return (c & ~7) | ((c ^ (c >> 3)) & 7); }

// The local pass's shared memory.
template <typename T, int S>
struct Input {
    static constexpr int CB = channels_of(S), VN = V16<T>::n, CH = CB / VN, BCH = S / VN;  // 16-byte chunks
    alignas(16) float4 d[kTile][CB];
    alignas(16) float b[2][kTile][S];
    uint4 x[2][kTile][CH], dt[2][kTile][CH], dy[2][kTile][CH], z[2][kTile][CH];
    uint4 bc[2][2 * kTile * BCH];
    alignas(16) float bias[CB];
};

// The number of the tile of first token t0 among the stored ones (-1: none is stored that starts before kTile).
__device__ __forceinline__ int place_of(int t0) { return (int)((unsigned)t0 / kTile) - 1; }

// Where a CTA stands: sequence, segment, its tokens [lo, hi), group, channels.
struct Where {
    int n, seg, lo, hi, eos, g, blk, cg0, c0;
};
template <typename T, int S>
__device__ __forceinline__ bool where(const BwdParams& q, Where& w) {
    const Params& p = q.f;
    const int nb = p.bpg * p.G, len = q.m * kTile;
    const int at = blockIdx.x / nb;
    w.blk = blockIdx.x % nb, w.g = w.blk / p.bpg, w.cg0 = (w.blk % p.bpg) * channels_of(S), w.c0 = w.g * p.CG + w.cg0;
    // the last sequence whose first segment is at or before `at`
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (max(0, min(__ldg(p.cu + mid), p.T)) / len + mid <= at) lo = mid;
        else hi = mid - 1;
    }
    int bos;
    bounds(p.cu, lo, p.T, bos, w.eos);
    const int k = at - (bos / len + lo);
    w.n = lo, w.seg = at;
    if (k < 0 || k > (w.eos - bos) / len) return false;
    w.lo = bos + k * len;
    w.hi = min(w.eos, w.lo + len);
    return w.lo < w.hi;
}

// A thread's share of a CTA's inputs: columns col .. col + VN - 1 of tokens row0, row0 + RS, .. of a
// tile.  Pointers and strides stay in the kernel's parameters: the walks need the registers.
template <typename T, int S, int NT>
struct Feed {
    using In = Input<T, S>;
    static constexpr int VN = In::VN, CH = In::CH, BCH = In::BCH, RS = NT / CH;
    static constexpr int NV = (kTile * CH + NT - 1) / NT, NB = (2 * kTile * BCH + NT - 1) / NT;
    static_assert(NT % CH == 0, "a thread keeps its columns");
    const BwdParams& q;
    int row0, ch, col, hi, c, g;
    bool cok;

    __device__ __forceinline__ Feed(const BwdParams& q_, const Where& w) : q(q_) {
        row0 = threadIdx.x / CH, ch = threadIdx.x % CH, col = ch * VN, hi = w.hi, c = w.c0 + col, g = w.g;
        cok = w.cg0 + col < q.f.CG;
    }
    // dt_bias of the CTA's channels; in place after the next barrier.
    __device__ __forceinline__ void columns(In& in, const Where& w) const {
        const Params& p = q.f;
        for (int i = threadIdx.x; i < In::CB; i += NT) {
            const bool ok = w.cg0 + i < p.CG;
            in.bias[i] = ok && p.bias ? __ldg(p.bias + w.c0 + i) : 0.f;
        }
    }
    __device__ __forceinline__ bool gate() const { return q.f.z != nullptr; }
    __device__ __forceinline__ bool has(int t0, int r) const {
        const int tt = row0 + r * RS;
        return tt < kTile && t0 + tt < hi && cok;
    }
    __device__ __forceinline__ void copy(In& in, int t0, int buf) const {
        const Params& p = q.f;
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int tt = row0 + r * RS;
            const int64_t t = t0 + tt;
            if (has(t0, r)) {
                copy16_async(&in.x[buf][tt][ch], static_cast<const T*>(p.x) + t * p.ldx + c);
                copy16_async(&in.dt[buf][tt][ch], static_cast<const T*>(p.dt) + t * p.lddt + c);
                copy16_async(&in.dy[buf][tt][ch], static_cast<const T*>(q.dy) + t * p.C + c);
                if (gate()) copy16_async(&in.z[buf][tt][ch], static_cast<const T*>(p.z) + t * p.ldz + c);
            }
        }
#pragma unroll
        for (int r = 0; r < NB; ++r) {
            const int v = threadIdx.x + NT * r, which = v / (kTile * BCH), k = v % (kTile * BCH);
            const int64_t t = t0 + k / BCH;
            const int e = g * S + (k % BCH) * VN;
            if (which < 2 && t < hi)
                copy16_async(&in.bc[buf][v], which ? static_cast<const T*>(p.Cm) + t * p.ldC + e : static_cast<const T*>(p.B) + t * p.ldB + e);
        }
    }
    // {d, d x, e, softplus'} and the fp32 B and C of the tile whose copies have arrived.
    __device__ __forceinline__ void prepare(In& in, int t0, int buf) const {
        const Params& p = q.f;
#pragma unroll
        for (int r = 0; r < NV; ++r) {
            const int tt = row0 + r * RS;
            if (tt >= kTile) continue;
            if (!has(t0, r)) {
#pragma unroll
                for (int e = 0; e < VN; ++e) in.d[tt][place(col + e)] = make_float4(0.f, 0.f, 0.f, 0.f);
                continue;
            }
            float2 xv[VN / 2], dv[VN / 2], ev[VN / 2], zv[VN / 2];
            unpack2(in.x[buf][tt][ch], xv);
            unpack2(in.dt[buf][tt][ch], dv);
            unpack2(in.dy[buf][tt][ch], ev);
            if (gate()) unpack2(in.z[buf][tt][ch], zv);
#pragma unroll
            for (int e = 0; e < VN / 2; ++e) {
                float2 d = __fadd2_rn(dv[e], *reinterpret_cast<const float2*>(&in.bias[col + 2 * e])), sig = both(1.f), u, s;
                if (p.softplus) {
                    const float2 v = d;
                    d = softplus2(v, u);
                    sig = sigmoid2(v, u);
                }
                const float2 dx = __fmul2_rn(d, xv[e]);
                const float2 g = gate() ? __fmul2_rn(ev[e], silu2(zv[e], s)) : ev[e];
                in.d[tt][place(col + 2 * e)] = make_float4(d.x, dx.x, g.x, sig.x);
                in.d[tt][place(col + 2 * e + 1)] = make_float4(d.y, dx.y, g.y, sig.y);
            }
        }
#pragma unroll
        for (int r = 0; r < NB; ++r) {
            const int v = threadIdx.x + NT * r, which = v / (kTile * BCH), k = v % (kTile * BCH);
            if (which < 2) {
                const bool ok = t0 + k / BCH < hi;
                float f[VN];
                unpack(in.bc[buf][v], f);
                float4* to = reinterpret_cast<float4*>(&in.b[which][k / BCH][(k % BCH) * VN]);
#pragma unroll
                for (int e = 0; e < VN; e += 4) to[e / 4] = ok ? make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
};

__device__ __forceinline__ void load_state(const float* p, float2 (&h)[2]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    h[0] = make_float2(u.x, u.y), h[1] = make_float2(u.z, u.w);
}
__device__ __forceinline__ void store_state(float* p, const float2 (&h)[2]) {
    *reinterpret_cast<float4*>(p) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
}
__device__ __forceinline__ float2 ex2_2(const float2& v) { return make_float2(ex2(v.x), ex2(v.y)); }

// ---------------------------------------------------------------- 1. local
// Every warp prepares and walks in turn: preparing on other warps, as 3 does, took as long (all
// of 8192 x 4096 x 16 within 0.3 %, 8 states 3 % longer), for the walk itself keeps the issue slots.
template <typename T, int S>
__global__ void __launch_bounds__(Geo<T, S, 4>::NT, 512 / Geo<T, S, 4>::NT) scan_local_kernel(const __grid_constant__ BwdParams q) {
    using F = Geo<T, S, 4>;
    constexpr int L = F::L;
    __shared__ Input<T, S> in;
    Where w;
    if (!where<T, S>(q, w)) return;
    const Params& p = q.f;
    const Feed<T, S, F::NT> feed(q, w);
    feed.copy(in, w.lo, 0);
    copy_commit();
    feed.columns(in, w);
    const int j = threadIdx.x % L, cl = threadIdx.x / L * 4;
    const bool ok = w.cg0 + cl < p.CG;  // all 4 or none: p.CG is a multiple of 8
    const int64_t C = p.C, own = ok ? (int64_t)(w.c0 + cl) * S + 4 * j : 0;
    float2 A2[4][2], h[4][2], G[4][2], P[4][2];
    float cum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        load4(p.A_log + own + (int64_t)(ok ? c : 0) * S, A2[c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            A2[c][i] = make_float2(a_log2(A2[c][i].x), a_log2(A2[c][i].y));
            h[c][i] = G[c][i] = both(0.f), P[c][i] = both(1.f);
        }
    }
    int at[4];  // this lane's channels in a row of in.d
#pragma unroll
    for (int c = 0; c < 4; ++c) at[c] = place(cl + c);
    int64_t tile = place_of(w.lo);
    __syncthreads();
    for (int t0 = w.lo, buf = 0; t0 < w.hi; t0 += kTile, buf ^= 1, ++tile) {
        copy_wait<0>();
        feed.prepare(in, t0, buf);
        __syncthreads();
        feed.copy(in, t0 + kTile, buf ^ 1);
        copy_commit();
        if (ok && t0 > w.lo) {
#pragma unroll
            for (int c = 0; c < 4; ++c) store_state(q.tiles + tile * C * S + own + c * S, h[c]);
            if (j == 0) *reinterpret_cast<float4*>(q.cum + tile * C + w.c0 + cl) = make_float4(cum[0], cum[1], cum[2], cum[3]);
        }
#pragma unroll 1
        for (int t = 0; t < kTile; ++t) {
            float2 b[2], k[2];
            load_state(&in.b[0][t][4 * j], b);
            load_state(&in.b[1][t][4 * j], k);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 v = in.d[t][at[c]];
                cum[c] = __fadd_rn(cum[c], v.x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 a = ex2_2(__fmul2_rn(both(v.x), A2[c][i]));
                    h[c][i] = __ffma2_rn(a, h[c][i], __fmul2_rn(both(v.y), b[i]));
                    P[c][i] = __fmul2_rn(P[c][i], a);
                    G[c][i] = __ffma2_rn(P[c][i], __fmul2_rn(both(v.z), k[i]), G[c][i]);
                }
            }
        }
        __syncthreads();
    }
    copy_wait<0>();
    if (!ok) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        store_state(q.seg_h + (int64_t)w.seg * C * S + own + c * S, h[c]);
        store_state(q.seg_g + (int64_t)w.seg * C * S + own + c * S, G[c]);
    }
    if (j == 0) *reinterpret_cast<float4*>(q.seg_d + (int64_t)w.seg * C + w.c0 + cl) = make_float4(cum[0], cum[1], cum[2], cum[3]);
}

// ---------------------------------------------------------------- 2. join
// A thread joins 4 states of one channel along one sequence: forwards (blockIdx.y 0) the start
// states, backwards (1) the end G's.  The loads do not depend on the chain and run ahead of it.
__global__ void __launch_bounds__(128) scan_join_kernel(const __grid_constant__ BwdParams q, int S) {
    const Params& p = q.f;
    const int64_t CS = (int64_t)p.C * S;
    const int blocks = (int)((CS / 4 + blockDim.x - 1) / blockDim.x), n = blockIdx.x / blocks;
    const int64_t i = ((int64_t)(blockIdx.x % blocks) * blockDim.x + threadIdx.x) * 4;
    if (i >= CS) return;
    const int c = (int)(i / S), len = q.m * kTile;
    const bool back = blockIdx.y;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int segs = (eos - bos + len - 1) / len;
    const int64_t first = bos / len + n;
    float2 A2[2], h[2] = {both(0.f), both(0.f)};
    load4(p.A_log + i, A2);
    A2[0] = make_float2(a_log2(A2[0].x), a_log2(A2[0].y)), A2[1] = make_float2(a_log2(A2[1].x), a_log2(A2[1].y));
    const float* from = back ? q.dhT : q.h0;
    if (from) load_state(from + n * CS + i, h);
    float* seg = back ? q.seg_g : q.seg_h;
    constexpr int U = 8;
    for (int k0 = 0; k0 < segs; k0 += U) {
        float2 s[U][2];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < segs) {
                const int64_t at = first + (back ? segs - 1 - k0 - u : k0 + u);
                load_state(seg + at * CS + i, s[u]);
                d[u] = q.seg_d[at * p.C + c];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k0 + u < segs) {
                const int64_t at = first + (back ? segs - 1 - k0 - u : k0 + u);
                store_state(seg + at * CS + i, h);
#pragma unroll
                for (int m = 0; m < 2; ++m) h[m] = __ffma2_rn(ex2_2(__fmul2_rn(both(d[u]), A2[m])), h[m], s[u][m]);
            }
    }
    if (back && q.dh0) store_state(q.dh0 + n * CS + i, h);
}

// ---------------------------------------------------------------- 3. grad
// Sum over the lanes of a channel in UP parts: with four lanes or more the last addition is left to
// the other warps (1 % of the whole gradient of 8192 tokens x 4096 channels x 16 states, 3 % of 4096 x
// 2048 x 32, fp32).
// Slot c of lane j holds channel c ^ (j & 1) of the lane's two: the first slot stays, the second
// goes to the neighbour, whose first it is, without selecting; further lanes add by a butterfly.
// Lane j ends with channel j & 1 of part j / (L / UP).
template <int L, int UP>
__device__ __forceinline__ float sum_states(const float (&v)[2]) {
    float s = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[1], 1));
#pragma unroll
    for (int off = 2; off < L / UP; off <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}
// Sum of a lane's four states over its lane group and its neighbour.  Pair slot m of group k holds pair
// m ^ (k & 1): the first slot stays, the second goes to the neighbour group.  The groups' sums are
// added up by the other warps, whose issue slots are fewer for it than the walkers' shuffles would be
// (with the whole sum here 8192 x 4096 x 16 took 8 % longer).
template <int L>
__device__ __forceinline__ float2 sum_neighbours(const float2 (&v)[2]) {
    constexpr uint32_t all = 0xffffffffu;
    return make_float2(__fadd_rn(v[0].x, __shfl_xor_sync(all, v[1].x, L)), __fadd_rn(v[0].y, __shfl_xor_sync(all, v[1].y, L)));
}

// Keeps the compiler from loading later tokens' values early: the states of a tile fill the registers.
__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

// The work per (token, channel) before and after a tile's walk is done beside it, on SIDE threads
// of their own: a thread takes 4 channels of tokens row0, row0 + RS, .. of every tile, prepares
// them for tile i + 1 while the walkers are at tile i, then waits for their sums and finishes it.
template <typename T> struct V4;
template <> struct V4<float> { using type = uint4; };
template <> struct V4<__nv_bfloat16> { using type = uint2; };
__device__ __forceinline__ void unpack4(const uint4& u, float2 (&v)[2]) { unpack2(u, v); }
__device__ __forceinline__ void unpack4(const uint2& u, float2 (&v)[2]) {
    v[0] = make_float2(bf_lo(u.x), bf_hi(u.x)), v[1] = make_float2(bf_lo(u.y), bf_hi(u.y));
}
__device__ __forceinline__ void copy4_async(uint4* to, const float* from) { copy16_async(to, from); }
__device__ __forceinline__ void copy4_async(uint2* to, const __nv_bfloat16* from) { copy8_async(to, from); }
__device__ __forceinline__ void store4_stream(float* to, const float2 (&v)[2]) {
    __stcs(reinterpret_cast<float4*>(to), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
}
__device__ __forceinline__ void store4_stream(__nv_bfloat16* to, const float2 (&v)[2]) {
    __nv_bfloat162 a = __float22bfloat162_rn(v[0]), b = __float22bfloat162_rn(v[1]);
    __stcs(reinterpret_cast<uint2*>(to), make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)));
}

template <typename T, int S>
struct GradMem {
    using F = Geo<T, S, 2>;
    using V = typename V4<T>::type;
    static constexpr int CB = F::CB, WALK = F::NT, SIDE = WALK < 128 ? 64 : 128, NT = WALK + SIDE;
    static constexpr int MINB = NT <= 128 ? 4 : 2;  // CTAs an SM shall hold
    static constexpr int CH = CB / 4, RS = SIDE / CH, NV = (kTile + RS - 1) / RS;
    static constexpr int NBC = 2 * kTile * S / 4;
    static constexpr int H = WALK == 128 ? kTile : kTile / 2;  // tokens whose states are in registers at a time
    static constexpr int PB = S == 16 || S == 32 ? 2 : 1;  // buffers of the lanes' dB and dC: with two, fewer than MINB CTAs find room
    // {d, d x, e, softplus'} of channel c at place(c); then B and C in fp32
    alignas(16) float4 d[2][kTile][CB];
    alignas(16) float b[2][2][kTile][S];
    static constexpr int UP = F::L < 4 ? 1 : 2;
    alignas(16) float uvy[2][3][kTile][UP][CB + (UP > 1 ? 16 : 4)];  // u, sum w A2, y in parts
    alignas(16) float4 bc[PB][kTile][WALK / 32][32];  // each lane's pair of dB and of dC, two groups of lanes added
    alignas(16) V x[2][kTile][CH], dt[2][kTile][CH], dy[2][kTile][CH], z[2][kTile][CH], in[2][NBC];
    // each walker's own: its segment's start states, the next tile's local ones, its states at the tile's start
    alignas(16) float4 seg[2][WALK];
    alignas(16) float4 tile[2][WALK];
    alignas(16) float4 h[2][H < kTile ? WALK : 1];
    static_assert(SIDE % CH == 0, "a thread keeps its columns");
};

// Two channels' states, their gradients and a tile's history need more registers than the work
// before and after: as in the forward, registers move to the walkers, no more than the CTA was
// launched with (128 a thread at two CTAs of 256 threads, 80 at two of 384; checked on the host).
// 8192 tokens x 4096 channels x 16 states, all kernels: 790 us at 80 and 176 registers, 790 at 88 and
// 168, 833 at 64 and 192, 902 at 56 and 200.  Before the sums went to the other warps, two CTAs an SM with
// a tile's history took 4 % less than with half a tile's, 6 % less than three with 112 registers and half a
// tile's, and 9 % less than every warp doing all phases in turn.
__host__ __device__ constexpr int regs_side(int walkers) { return walkers == 128 ? 80 : 48; }
__host__ __device__ constexpr int regs_walk(int walkers) { return walkers == 128 ? 176 : 96; }

template <typename T, int S>
__global__ void __launch_bounds__(GradMem<T, S>::NT, GradMem<T, S>::MINB) scan_grad_kernel(const __grid_constant__ BwdParams q) {
    using M = GradMem<T, S>;
    using F = Geo<T, S, 2>;
    constexpr int L = F::L, CB = F::CB, WALK = M::WALK, SIDE = M::SIDE, NT = M::NT;
    constexpr int kFull = 1, kDone = 3, kLeft = 5, kSums = 6;  // named barriers, the first two one per buffer
    extern __shared__ __align__(16) unsigned char raw[];
    M& sm = *reinterpret_cast<M*>(raw);
    Where w;
    const bool some = where<T, S>(q, w);
    const Params& p = q.f;
    const int64_t C = p.C;
    if (!some) {  // no segment of this number: its parts of the sums are zero
        const int64_t at = (int64_t)w.seg * C + w.c0, n = min(CB, p.CG - w.cg0);
        for (int i = threadIdx.x; i < n * S; i += NT) q.seg_g[at * S + i] = 0.f;
        for (int i = threadIdx.x; i < n; i += NT) q.pD[at + i] = q.pb[at + i] = 0.f;
        return;
    }
    const int tiles = (w.hi - w.lo + kTile - 1) / kTile;

    if (threadIdx.x >= WALK) {
        if constexpr (M::SIDE == 128) regs_less<regs_side(WALK)>();
        const int tid = threadIdx.x - WALK, row0 = tid / M::CH, ch = tid % M::CH, col = 4 * ch;
        const bool cok = w.cg0 + col < p.CG, gate = p.z != nullptr;
        const int c = w.c0 + col;
        auto has = [&](int t0, int r) { return row0 + r * M::RS < kTile && t0 + row0 + r * M::RS < w.hi && cok; };
        auto copy = [&](int t0, int buf) {
#pragma unroll
            for (int r = 0; r < M::NV; ++r) {
                const int tt = row0 + r * M::RS;
                const int64_t t = t0 + tt;
                if (has(t0, r)) {
                    copy4_async(&sm.x[buf][tt][ch], static_cast<const T*>(p.x) + t * p.ldx + c);
                    copy4_async(&sm.dt[buf][tt][ch], static_cast<const T*>(p.dt) + t * p.lddt + c);
                    copy4_async(&sm.dy[buf][tt][ch], static_cast<const T*>(q.dy) + t * p.C + c);
                    if (gate) copy4_async(&sm.z[buf][tt][ch], static_cast<const T*>(p.z) + t * p.ldz + c);
                }
            }
            for (int v = tid; v < M::NBC; v += SIDE) {
                const int which = v / (kTile * S / 4), k = v % (kTile * S / 4);
                const int64_t t = t0 + k / (S / 4);
                const int e = w.g * S + k % (S / 4) * 4;
                if (t < w.hi)
                    copy4_async(&sm.in[buf][v], which ? static_cast<const T*>(p.Cm) + t * p.ldC + e : static_cast<const T*>(p.B) + t * p.ldB + e);
            }
            copy_commit();
        };
        float2 D[2], sD[2], sb[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            D[e] = cok && p.D ? make_float2(__ldg(p.D + c + 2 * e), __ldg(p.D + c + 2 * e + 1)) : both(0.f);
            sD[e] = sb[e] = both(0.f);
        }
        auto prepare = [&](int t0, int buf) {
#pragma unroll
            for (int r = 0; r < M::NV; ++r) {
                const int tt = row0 + r * M::RS;
                if (tt >= kTile) continue;
                if (!has(t0, r)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sm.d[buf][tt][place(col + e)] = make_float4(0.f, 0.f, 0.f, 0.f);
                    continue;
                }
                float2 xv[2], dv[2], ev[2], zv[2];
                unpack4(sm.x[buf][tt][ch], xv);
                unpack4(sm.dt[buf][tt][ch], dv);
                unpack4(sm.dy[buf][tt][ch], ev);
                if (gate) unpack4(sm.z[buf][tt][ch], zv);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 bias = p.bias ? make_float2(__ldg(p.bias + c + 2 * e), __ldg(p.bias + c + 2 * e + 1)) : both(0.f);
                    float2 d = __fadd2_rn(dv[e], bias), sig = both(1.f), u, s;
                    if (p.softplus) {
                        const float2 v = d;
                        d = softplus2(v, u);
                        sig = sigmoid2(v, u);
                    }
                    const float2 dx = __fmul2_rn(d, xv[e]);
                    const float2 g = gate ? __fmul2_rn(ev[e], silu2(zv[e], s)) : ev[e];
                    sm.d[buf][tt][place(col + 2 * e)] = make_float4(d.x, dx.x, g.x, sig.x);
                    sm.d[buf][tt][place(col + 2 * e + 1)] = make_float4(d.y, dx.y, g.y, sig.y);
                }
            }
            for (int v = tid; v < M::NBC; v += SIDE) {
                const int k = v % (kTile * S / 4);
                float2 f[2];
                unpack4(sm.in[buf][v], f);
                reinterpret_cast<float4*>(&sm.b[buf][0][0][0])[v] =
                    t0 + k / (S / 4) < w.hi ? make_float4(f[0].x, f[0].y, f[1].x, f[1].y) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            bar_arrive(kFull + buf, NT);
        };
        auto finish = [&](int t0, int buf) {
            // dB and dC: PT threads add up the warps' groups of one token and pair of states
            const auto& bc = sm.bc[M::PB > 1 ? buf : 0];
            constexpr int OUT = kTile * 2 * L, PT = SIDE > OUT ? SIDE / OUT : 1, NW = WALK / 32 / PT;
#pragma unroll 1
            for (int f = tid; f < OUT * PT; f += SIDE) {
                const int pm = f % (2 * L) / L, j = f % L, part = f / (2 * L) % PT, tt = f / (2 * L * PT);
                float2 b2 = both(0.f), c2 = both(0.f);
#pragma unroll
                for (int i = 0; i < NW; ++i)
#pragma unroll
                    for (int k = 0; k < 32 / L; k += 2) {
                        const float4 v = bc[tt][part * NW + i][(k + pm) * L + j];
                        b2 = __fadd2_rn(b2, make_float2(v.x, v.y)), c2 = __fadd2_rn(c2, make_float2(v.z, v.w));
                    }
#pragma unroll
                for (int off = 1; off < PT; off <<= 1) {
                    const float2 u = make_float2(__shfl_xor_sync(0xffffffffu, b2.x, 2 * L * off), __shfl_xor_sync(0xffffffffu, b2.y, 2 * L * off));
                    const float2 v = make_float2(__shfl_xor_sync(0xffffffffu, c2.x, 2 * L * off), __shfl_xor_sync(0xffffffffu, c2.y, 2 * L * off));
                    b2 = __fadd2_rn(b2, u), c2 = __fadd2_rn(c2, v);
                }
                if (part == 0 && t0 + tt < w.hi) {
                    float* to = q.bc + ((int64_t)w.blk * p.T + t0 + tt) * 2 * S + 4 * j + 2 * pm;
                    *reinterpret_cast<float2*>(to) = b2, *reinterpret_cast<float2*>(to + S) = c2;
                }
            }
            if (M::PB == 1 && t0 > w.lo) bar_arrive(kLeft, NT);
#pragma unroll
            for (int r = 0; r < M::NV; ++r) {
                if (!has(t0, r)) break;
                const int tt = row0 + r * M::RS;
                const int64_t to = (int64_t)(t0 + tt) * C + c;
                float2 xv[2], odx[2], odt[2], odz[2];
                unpack4(sm.x[buf][tt][ch], xv);
                auto sum_of = [&](int which, int e) {
                    float2 v = *reinterpret_cast<const float2*>(&sm.uvy[buf][which][tt][0][col + 2 * e]);
                    if constexpr (M::UP > 1) v = __fadd2_rn(v, *reinterpret_cast<const float2*>(&sm.uvy[buf][which][tt][1][col + 2 * e]));
                    return v;
                };
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 v0 = sm.d[buf][tt][place(col + 2 * e)], v1 = sm.d[buf][tt][place(col + 2 * e + 1)];
                    const float2 d = make_float2(v0.x, v1.x), g = make_float2(v0.z, v1.z), sig = make_float2(v0.w, v1.w);
                    const float2 u = sum_of(0, e), v = __fmul2_rn(sum_of(1, e), both(kLn2));
                    odx[e] = __ffma2_rn(d, u, __fmul2_rn(D[e], g));
                    // a masked token (dt = -inf, slope 0) gets 0, though a decay past fp32 may have made its dd infinite
                    const float2 dd = __ffma2_rn(xv[e], u, v);
                    odt[e] = make_float2(sig.x != 0.f ? __fmul_rn(dd.x, sig.x) : 0.f, sig.y != 0.f ? __fmul_rn(dd.y, sig.y) : 0.f);
                    sD[e] = __ffma2_rn(g, xv[e], sD[e]);
                    sb[e] = __fadd2_rn(sb[e], odt[e]);
                }
                store4_stream(static_cast<T*>(q.dx) + to, odx);
                store4_stream(static_cast<T*>(q.ddt) + to, odt);
                if (gate) {
                    float2 ev[2], zv[2];
                    unpack4(sm.dy[buf][tt][ch], ev), unpack4(sm.z[buf][tt][ch], zv);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float2 s;
                        const float2 y = __ffma2_rn(D[e], xv[e], sum_of(2, e));
                        silu2(zv[e], s);
                        const float2 slope = __fmul2_rn(s, __ffma2_rn(zv[e], __ffma2_rn(s, both(-1.f), both(1.f)), both(1.f)));
                        odz[e] = __fmul2_rn(__fmul2_rn(ev[e], y), slope);
                    }
                    store4_stream(static_cast<T*>(q.dz) + to, odz);
                }
            }
        };
        auto at = [&](int i) { return w.lo + (tiles - 1 - i) * kTile; };  // the i-th tile walked
        copy(at(0), 0);
        copy_wait<0>();
        prepare(at(0), 0);
        if (tiles > 1) copy(at(1), 1);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
            const int buf = i & 1;
            if (i + 1 < tiles) {
                copy_wait<0>();
                prepare(at(i + 1), buf ^ 1);
            }
            bar_sync(kDone + buf, NT);
            finish(at(i), buf);
            if (i + 2 < tiles) copy(at(i + 2), buf);
        }
        // the columns' sums over these threads, in the order of their rows
        float2* sums = reinterpret_cast<float2*>(&sm.uvy[0][0][0][0][0]);
        bar_sync(kSums, SIDE);
#pragma unroll
        for (int e = 0; e < 2; ++e) sums[(2 * tid + e) * 2] = sD[e], sums[(2 * tid + e) * 2 + 1] = sb[e];
        bar_sync(kSums, SIDE);
        for (int f = tid; f < 2 * CB; f += SIDE) {
            const int k = f % CB, e = k % 4 / 2;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < (M::RS < kTile ? M::RS : kTile); ++r) {
                const float2 v = sums[(2 * (r * M::CH + k / 4) + e) * 2 + (f >= CB)];
                s = __fadd_rn(s, k & 1 ? v.y : v.x);
            }
            if (w.cg0 + k < p.CG) (f < CB ? q.pD : q.pb)[(int64_t)w.seg * C + w.c0 + k] = s;
        }
        return;
    }

    if constexpr (M::SIDE == 128) regs_more<regs_walk(WALK)>();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool gate = p.z != nullptr;
    const int j = tid % L, jq = j & 1, cl = tid / L * 2, pm = tid / L & 1;
    const bool ok = w.cg0 + cl < p.CG;
    const int64_t own = ok ? (int64_t)(w.c0 + cl) * S + 4 * j : 0;
    // slot c: channel cl + (c ^ jq); pair slot i: states 4 j + 2 (i ^ pm) and the next one
    const int at0 = place(cl + jq), at1 = place(cl + (jq ^ 1));
    const int64_t so0 = own + (ok ? jq : 0) * S, so1 = own + (ok ? jq ^ 1 : 0) * S;
    const int first = place_of(w.lo);
    auto copy_tile = [&](int k) {  // the local states at tile k's start
        const float* from = q.tiles + (int64_t)(first + k) * C * S;
        if (k > 0) copy16_async(&sm.tile[0][tid], from + so0), copy16_async(&sm.tile[1][tid], from + so1);
        copy_commit();
    };
    copy_tile(tiles - 1);
    sm.seg[0][tid] = *reinterpret_cast<const float4*>(q.seg_h + (int64_t)w.seg * C * S + so0);
    sm.seg[1][tid] = *reinterpret_cast<const float4*>(q.seg_h + (int64_t)w.seg * C * S + so1);
    auto cum_of = [&](int k, int c) { return ok && k > 0 ? q.cum[(int64_t)(first + k) * C + w.c0 + cl + (c ^ jq)] : 0.f; };
    float cum[2] = {cum_of(tiles - 1, 0), cum_of(tiles - 1, 1)};
    auto load_pairs = [&](const float* from, float2 (&v)[2]) {
        float2 t[2];
        load_state(from, t);
        v[0] = pm ? t[1] : t[0], v[1] = pm ? t[0] : t[1];
    };
    float2 A2[2][2], G[2][2], dA[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        load_pairs(p.A_log + (c ? so1 : so0), A2[c]);
        load_pairs(q.seg_g + (int64_t)w.seg * C * S + (c ? so1 : so0), G[c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            A2[c][i] = make_float2(a_log2(A2[c][i].x), a_log2(A2[c][i].y));
            if (!ok) A2[c][i] = G[c][i] = both(0.f);  // the values of another group's channel stay out of this one's dB and dC
            dA[c][i] = both(0.f);
        }
    }
    for (int k = tiles - 1, buf = 0; k >= 0; --k, buf ^= 1) {
        copy_wait<0>();
        float2 h[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // the tile's start: its segment's start state, decayed, plus the local state
            const float4 v = sm.seg[c][tid], u = sm.tile[c][tid];
            h[c][0] = pm ? make_float2(v.z, v.w) : make_float2(v.x, v.y), h[c][1] = pm ? make_float2(v.x, v.y) : make_float2(v.z, v.w);
            const float2 s[2] = {pm ? make_float2(u.z, u.w) : make_float2(u.x, u.y), pm ? make_float2(u.x, u.y) : make_float2(u.z, u.w)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (k) h[c][i] = __ffma2_rn(ex2_2(__fmul2_rn(both(cum[c]), A2[c][i])), h[c][i], s[i]);
                if (!ok) h[c][i] = both(0.f);
            }
        }
        cum[0] = cum_of(k - 1, 0), cum[1] = cum_of(k - 1, 1);
        copy_tile(k - 1);
        bar_sync(kFull + buf, NT);
        if (M::PB == 1 && k < tiles - 1) bar_sync(kLeft, NT);
        auto& bc = sm.bc[M::PB > 1 ? buf : 0];
        auto& uvy = sm.uvy[buf];

        auto pairs = [&](int which, int t, float2 (&v)[2]) {
            const float2* from = reinterpret_cast<const float2*>(&sm.b[buf][which][t][4 * j]);
            v[0] = from[pm], v[1] = from[pm ^ 1];
        };
        auto step = [&](int t, const float2 (&from)[2][2], float2 (&to)[2][2]) {
            float2 b[2];
            fence();
            pairs(0, t, b);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float2 v = *reinterpret_cast<const float2*>(&sm.d[buf][t][c ? at1 : at0]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    to[c][i] = from[c][i];
                    advance(to[c][i], A2[c][i], both(v.x), both(v.y), b[i]);
                }
            }
        };
        // H tokens at a time: with H = kTile / 2 the second half of the tile, then, from its start again, the first
        constexpr int H = M::H;
        if constexpr (H < kTile) {
#pragma unroll
            for (int c = 0; c < 2; ++c) sm.h[c][tid] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
#pragma unroll
            for (int t = 0; t < H; ++t) step(t, h, h);
        }
#pragma unroll 1
        for (int half = kTile - H; half >= 0; half -= H) {
            float2 old[H + 1][2][2];  // the states before each of these tokens, and behind the last
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) old[0][c][i] = h[c][i];
#pragma unroll
            for (int t = 0; t < H; ++t) step(half + t, old[t], old[t + 1]);
#pragma unroll
            for (int t = H - 1; t >= 0; --t) {
                float2 b[2], kc[2], sB[2], sC[2];
                float us[2], vs[2], ys[2];
                fence();
                pairs(0, half + t, b);
                pairs(1, half + t, kc);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float4 v = sm.d[buf][half + t][c ? at1 : at0];
                    float2 u, x, y;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 a = ex2_2(__fmul2_rn(both(v.x), A2[c][i]));
                        const float2 g = __ffma2_rn(both(v.z), kc[i], G[c][i]), ht = old[t + 1][c][i];
                        y = i ? __ffma2_rn(ht, kc[i], y) : __fmul2_rn(ht, kc[i]);
                        sC[i] = c ? __ffma2_rn(ht, both(v.z), sC[i]) : __fmul2_rn(ht, both(v.z));
                        u = i ? __ffma2_rn(g, b[i], u) : __fmul2_rn(g, b[i]);
                        sB[i] = c ? __ffma2_rn(g, both(v.y), sB[i]) : __fmul2_rn(g, both(v.y));
                        G[c][i] = __fmul2_rn(a, g);
                        const float2 wv = __fmul2_rn(G[c][i], old[t][c][i]);
                        x = i ? __ffma2_rn(wv, A2[c][i], x) : __fmul2_rn(wv, A2[c][i]);
                        dA[c][i] = __ffma2_rn(wv, both(v.x), dA[c][i]);
                    }
                    us[c] = __fadd_rn(u.x, u.y), vs[c] = __fadd_rn(x.x, x.y), ys[c] = __fadd_rn(y.x, y.y);
                }
                constexpr int LP = L / M::UP;  // lanes of a part; the first two of them keep it
                const float u = sum_states<L, M::UP>(us), v = sum_states<L, M::UP>(vs);
                if (j % LP < 2) uvy[0][half + t][j / LP][cl + jq] = u, uvy[1][half + t][j / LP][cl + jq] = v;
                if (gate) {
                    const float y = sum_states<L, M::UP>(ys);
                    if (j % LP < 2) uvy[2][half + t][j / LP][cl + jq] = y;
                }
                const float2 db = sum_neighbours<L>(sB), dc = sum_neighbours<L>(sC);
                bc[half + t][warp][lane] = make_float4(db.x, db.y, dc.x, dc.y);
            }
            if constexpr (H < kTile)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float4 u = sm.h[c][tid];
                    h[c][0] = make_float2(u.x, u.y), h[c][1] = make_float2(u.z, u.w);
                }
        }
        bar_arrive(kDone + buf, NT);
    }
    copy_wait<0>();
    if (ok) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int i = 0; i < 2; ++i) dA[c][i] = __fmul2_rn(__fmul2_rn(dA[c][i], A2[c][i]), both(kLn2));
            const float2 v[2] = {pm ? dA[c][1] : dA[c][0], pm ? dA[c][0] : dA[c][1]};
            store_state(q.seg_g + (int64_t)w.seg * C * S + (c ? so1 : so0), v);
        }
    }
}

// ---------------------------------------------------------------- 4. sums
// Sums of rows: dB and dC of every covered token over the channel blocks of its group (the first
// `nbc` CTAs), dA_log [C, S], dD and ddt_bias [C] over the segments.  A CTA takes 16 neighbouring
// float4 columns; thread (slice, column) adds rows slice, slice + 16, .., then a thread per column
// adds the slices in order: 16 times the loads in flight of one thread a column.
template <typename T, int S>
__global__ void __launch_bounds__(256) scan_sums_kernel(const __grid_constant__ BwdParams q, unsigned nbc, int segs) {
    __shared__ float4 part[16][16];
    const Params& p = q.f;
    const int x = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const bool isbc = blockIdx.x < nbc;
    const int64_t col = (isbc ? blockIdx.x : blockIdx.x - nbc) * (int64_t)16 + x;
    const int64_t per = (int64_t)p.T * 2 * S / 4, nA = (int64_t)p.C * S / 4;  // float4 columns of a group, of dA
    const float4* src = nullptr;
    int64_t step = 0, t = 0;
    int rows = 0, g = 0;
    if (isbc) {
        g = (int)(col / per), t = col % per * 4 / (2 * S);
        if (g < p.G && t < max(0, min(__ldg(p.cu + p.N), p.T)))
            src = reinterpret_cast<const float4*>(q.bc) + (int64_t)g * p.bpg * per + col % per, step = per, rows = p.bpg;
    } else if (col < nA) {
        src = reinterpret_cast<const float4*>(q.seg_g) + col, step = nA, rows = segs;
    } else if (col < nA + p.C / 2) {
        const int64_t c = col - nA, half = p.C / 4;
        if (c < half ? q.dD != nullptr : q.dbias != nullptr)
            src = reinterpret_cast<const float4*>(c < half ? q.pD : q.pb) + c % half, step = half, rows = segs;
    }
    const bool any = src != nullptr;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v) { s.x = __fadd_rn(s.x, v.x), s.y = __fadd_rn(s.y, v.y), s.z = __fadd_rn(s.z, v.z), s.w = __fadd_rn(s.w, v.w); };
#pragma unroll 4
    for (int r = slice; r < rows; r += 16) add(src[r * step]);
    part[slice][x] = s;
    __syncthreads();
    if (slice || !any) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) add(part[i][x]);
    if (isbc) {
        const int e = (int)(col % per * 4 % (2 * S));
        T* out = static_cast<T*>(e < S ? q.dB : q.dC) + (t * p.G + g) * S + (e < S ? e : e - S);
        store1(out, s.x), store1(out + 1, s.y), store1(out + 2, s.z), store1(out + 3, s.w);
    } else {
        float* out = col < nA ? q.dA + col * 4 : col - nA < p.C / 4 ? q.dD + (col - nA) * 4 : q.dbias + (col - nA - p.C / 4) * 4;
        out[0] = s.x, out[1] = s.y, out[2] = s.z, out[3] = s.w;
    }
}

struct Layout {
    size_t tiles, cum, seg_h, seg_g, seg_d, bc, pD, pb, total;  // offsets in floats
    int bpg, m;
    long long segs;
};
Layout layout(const gdn_scan_shape* s) {
    const int cb = channels_of(s->S), cg = s->C / s->G;
    Layout l;
    l.bpg = (cg + cb - 1) / cb;
    // Tiles per segment: long segments save traffic and joins, short ones give a small batch CTAs
    // to run side by side.  us at 2 / 4 / 8 / 16, bf16, 16 states: 512 tokens x 512 channels 29 / 30 / 42 / 67,
    // 2048 x 1024 87 / 77 / 77 / 85, 2048 x 2048 151 / 130 / 124 / 134, 16384 x 1024 601 / 487 / 435 / 419.
    // Counted: the segments that the tokens make, and at most as many for the sequences' ragged ends; more
    // sequences are empty or one segment each whatever m is.
    auto ctas = [&](int m) {
        const long long full = s->T_total / (m * kTile);
        return (full + (s->N < full ? s->N : full)) * s->G * l.bpg;
    };
    // In waves of the CTAs that the GPU holds (fewer, and 16 lose to the last wave: 4096 x 4096 x 8, 3.6
    // waves at 16, 325 us, 317 at 8).
    const long long wave = kSMs * (s->S == 8 ? 4 : 2);
    l.m = ctas(16) >= 6 * wave ? 16 : ctas(8) >= 2 * wave ? 8 : ctas(4) >= wave ? 4 : 2;
    l.segs = (long long)s->T_total / (l.m * kTile) + s->N;
    const size_t c = s->C, cs = c * s->S, n = (size_t)l.segs, tiles = s->T_total / kTile;
    l.tiles = 0;
    l.cum = l.tiles + tiles * cs;
    l.seg_h = l.cum + tiles * c;
    l.seg_g = l.seg_h + n * cs;
    l.seg_d = l.seg_g + n * cs;
    l.bc = l.seg_d + n * c;
    l.pD = l.bc + (size_t)s->G * l.bpg * s->T_total * 2 * s->S;
    l.pb = l.pD + n * c;
    l.total = l.pb + n * c;
    return l;
}

template <typename T, int S>
gdn_status launch(cudaStream_t s, const BwdParams& q, long long segs) {
    const Params& p = q.f;
    const long long ctas = segs * p.G * p.bpg, bc = ((long long)p.T * p.G * 2 * S / 4 + 15) / 16;
    const long long par = ((long long)p.C * (S + 2) / 4 + 15) / 16;
    const long long joins = ((long long)p.C * S / 4 + 127) / 128 * p.N;
    if (ctas >= (1LL << 31) || bc + par >= (1LL << 31) || joins >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    constexpr size_t smem = sizeof(GradMem<T, S>);
    if constexpr (GradMem<T, S>::SIDE == 128) {
        using M = GradMem<T, S>;
        static std::atomic<int> known{0};
        const gdn_status st = check_registers(scan_grad_kernel<T, S>, M::NT, regs_side(M::WALK) * M::SIDE + regs_walk(M::WALK) * M::WALK, known);
        if (st != GDN_OK) return st;
    }
    if constexpr (smem > 48 * 1024) {
        if (cudaFuncSetAttribute(scan_grad_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return GDN_ERR_CUDA;
    }
    if (p.N > 0) {
        if (p.T > 0) scan_local_kernel<T, S><<<(unsigned)ctas, Geo<T, S, 4>::NT, 0, s>>>(q);
        scan_join_kernel<<<dim3((unsigned)joins, 2), 128, 0, s>>>(q, S);
        if (p.T > 0) scan_grad_kernel<T, S><<<(unsigned)ctas, GradMem<T, S>::NT, smem, s>>>(q);
    }
    scan_sums_kernel<T, S><<<(unsigned)(bc + par), 256, 0, s>>>(q, (unsigned)bc, p.T > 0 ? (int)segs : 0);
    return launch_status();
}
template <typename T>
gdn_status by_states(int S, cudaStream_t s, const BwdParams& q, long long segs) {
    switch (S) {
        case 8: return launch<T, 8>(s, q, segs);
        case 16: return launch<T, 16>(s, q, segs);
        case 32: return launch<T, 32>(s, q, segs);
        case 64: return launch<T, 64>(s, q, segs);
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
    const Layout l = layout(shape);
    if (!workspace || !aligned16(workspace) || workspace_bytes < l.total * sizeof(float)) return GDN_ERR_WORKSPACE;
    float* w = static_cast<float*>(workspace);
    BwdParams q{};
    scan::Params& p = q.f;
    p.N = shape->N, p.T = shape->T_total, p.C = shape->C, p.G = shape->G, p.CG = shape->C / shape->G, p.bpg = l.bpg;
    p.softplus = shape->dt_softplus;
    p.x = x, p.dt = dt, p.z = z, p.B = B, p.Cm = Cm;
    p.ldx = shape->ldx, p.lddt = shape->lddt, p.ldz = shape->ldz, p.ldB = shape->ldB, p.ldC = shape->ldC;
    p.A_log = A_log, p.D = D, p.bias = dt_bias, p.cu = cu_seqlens;
    q.m = l.m, q.h0 = init_state, q.dhT = d_final_state, q.dy = d_y;
    q.dx = dx, q.ddt = ddt, q.dz = dz, q.dB = dB, q.dC = dC;
    q.dA = dA_log, q.dD = dD, q.dbias = ddt_bias, q.dh0 = d_init_state;
    q.tiles = w + l.tiles, q.cum = w + l.cum, q.seg_h = w + l.seg_h, q.seg_g = w + l.seg_g, q.seg_d = w + l.seg_d;
    q.bc = w + l.bc, q.pD = w + l.pD, q.pb = w + l.pb;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return shape->dtype == GDN_BF16 ? by_states<__nv_bfloat16>(shape->S, s, q, l.segs) : by_states<float>(shape->S, s, q, l.segs);
}
