// gdn_scan.cu -- the selective state space scan: prompts (and the trainer's forward) and
// single tokens.  The arithmetic is in gdn_scan.cuh.
#include "gdn_async.cuh"
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

// The sequence of rank `rank` by length, the longest first (ties by number).  As soon as an SM gets
// more than one CTA, the longest walks must neither start last nor share an SM: 16 ragged prompts,
// 16384 x 8192 x 16, take 640 us in order of number and 536 in order of length (one channel a lane
// 601 and 564); two CTAs an SM, all resident from the start (8000 x 2048 x 16), 188 and 149.
// A CTA's N^2 comparisons have to be few against its walk of T / N tokens: ranked and not, 256
// sequences take 473 and 220 us at 4096 x 8192 x 16, 298 and 317 at 65536 x 1024, 546 and 665 at
// 131072 x 1024; hence N^3 <= 256 T.
constexpr int kRanked = 256;
__device__ __forceinline__ int ranked(const Params& p, int rank, int threads) {
    __shared__ int len[kRanked], found;
    for (int i = threadIdx.x; i < p.N; i += threads) {
        int bos, eos;
        bounds(p.cu, i, p.T, bos, eos);
        len[i] = eos - bos;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.N; i += threads) {
        const int mine = len[i];
        int before = 0;
        for (int k = 0; k < p.N; ++k) before += len[k] > mine || (len[k] == mine && k < i);
        if (before == rank) found = i;
    }
    __syncthreads();
    return found;
}

// Prompts.  A CTA walks one sequence over CB channels in tiles of TT tokens.  The phases before
// and after the walk run beside it, on other warps, a tile ahead and a tile behind:
//   * preparers, the work per (token, channel), 16-byte chunks of x and dt: d = softplus(dt + bias)
//     and d x, and B and C in fp32, of tile i + 1 to shared memory;
//   * walkers, the recurrence over tile i, a lane 8 states of Q channels (L = S / 8 lanes a
//     channel), sum_s h C in UP parts to shared memory;
//   * finishers: the parts' sum, skip term, gate and 16-byte stores of tile i - 1.
// They meet at named barriers: full (tile prepared), free (its d, B, C read), done (its sums
// written), left (its sums read), one of each per buffer; every side passes each barrier the
// same number of times.  Preparers and finishers copy their own inputs, asynchronously, a tile
// ahead, and read back only chunks that they copied themselves.
//
// What bounds it: with few CTAs the walkers' latency; with many the issue slots (63 % busy) and the
// path from shared memory into registers (128 bytes a cycle, whether lanes share an address or not; B and
// C take 64 bytes a lane and token), 70 % busy with Q = 1 and 61 % with Q = 2: neither is full.  The step
// alone (per two states 4 packed products or fmas and 2 exponentials, in registers) was measured at 6.8 T
// states/s on this GPU, the exponentials alone at 10 T and the fmas at 9.6 T; the kernel reaches 4.1 T at 16
// states, 4.5 T at 64.  The difference is loading the operands and the phases around the walk, and for ragged
// prompts the last ones to end.  ns a token of all CTAs, 2048 tokens, 16 states, bf16, at 1 / 2 / 3 / 4 / 8 /
// 16 blocks of 64 channels an SM: Q = 1 60 / 93 / 130 / 173 / 327 / 638, Q = 2 102 / 103 / 167 / 168 / 314 /
// 601; 64 states, 8 blocks of 16 channels: 357 and 277.
template <typename T, int S, int Q>
struct FwdTile {
    static constexpr int L = S / 8, CB = Q * (S <= 16 ? 64 : 1024 / S), VN = V16<T>::n, TT = 16 / Q;
    static constexpr int WALK = CB / Q * L, SIDE = 64, NT = WALK + 2 * SIDE;
    // CTAs an SM shall hold.  With 2 and the registers that this leaves, full SMs lose 4 to 6 % (the 16
    // prompts above, Q = 1: 564 and 588 us; Q = 2: 536 and 570), with 4 1 to 5 % (571; 560).
    static constexpr int MINB = 3;
    static constexpr int CH = CB / VN, NV = (TT * CH + SIDE - 1) / SIDE, RS = SIDE / CH;
    static constexpr int BCH = S / VN, NB = (2 * TT * BCH + SIDE - 1) / SIDE;
    // {d, d x} of channel c at c float2s plus one 16-byte gap per 16 channels: the chunk-wise
    // stores and the lanes' loads are both free of bank conflicts.
    static constexpr int ROW = CB + (CB / 16) * 2;
    static constexpr int YROW = CB + (L > 1 ? 32 / L : 0);  // the lanes' stores of L tokens miss each other's banks
    static constexpr int ST = 2;                    // tiles of inputs in flight or in use
    alignas(16) float2 d[2][TT][ROW];
    // States 8 j + 4 k .. of B (C) at float4 k L + j: the L lanes' loads touch consecutive chunks
    // (in order of states, 8 lanes would meet in the same banks: 64 states 6 % slower).
    float4 b[2][2][TT][2 * L];
    // Parts of a sum, whose last addition is the finishers' (the 16 prompts: 542 us with it in the walk, 536
    // so; with one channel a lane the room for two parts would cost fp32 a CTA an SM).
    static constexpr int UP = Q > 1 ? 2 : 1;
    alignas(16) float y[2][TT][UP][YROW];
    uint4 x[ST][TT][CH], dt[ST][TT][CH], bc[ST][2 * TT * BCH];  // preparers'
    uint4 x2[ST][TT][CH], z[ST][TT][CH];                        // finishers'
    static_assert(SIDE % CH == 0, "a thread keeps its columns");
    static_assert(Q == 1 || (WALK == 128 && 2 * SIDE == 128), "registers move between warpgroups");
};


// With two channels a lane the walkers need more registers than the others.  A thread is launched
// with 80 (at three CTAs of 256 threads); 128 threads go down to 64, 128 up to 96, no more than the
// CTA holds (checked on the host).  Without: 576 us for the 16 prompts instead of 536; 48 and 112: 558;
// 56 and 104: 526.
constexpr int kRegsSide = 64, kRegsWalk = 96;

template <typename T, int S, int Q>
__global__ void __launch_bounds__(FwdTile<T, S, Q>::NT, FwdTile<T, S, Q>::MINB) scan_fwd_kernel(const __grid_constant__ Params p) {
    using F = FwdTile<T, S, Q>;
    constexpr int L = F::L, CB = F::CB, TT = F::TT, VN = F::VN, CH = F::CH, NV = F::NV, RS = F::RS, BCH = F::BCH, NB = F::NB, ST = F::ST;
    constexpr int kFull = 1, kFree = 3, kDone = 5, kLeft = 7, kPair = F::WALK + F::SIDE;
    extern __shared__ __align__(16) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const int nb = p.bpg * p.G;
    const int at = blockIdx.x / nb, blk = blockIdx.x % nb;
    const int n = p.ranked ? ranked(p, at, F::NT) : at;
    const int g = blk / p.bpg, cg0 = (blk % p.bpg) * CB, c0 = g * p.CG + cg0;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int tiles = (eos - bos + TT - 1) / TT;

    if (threadIdx.x >= F::WALK) {
        if constexpr (Q > 1) regs_less<kRegsSide>();
        const bool first = threadIdx.x < F::WALK + F::SIDE;
        const int tid = (threadIdx.x - F::WALK) % F::SIDE;
        const int row0 = tid / CH, ch = tid % CH, col = ch * VN;
        const bool cok = cg0 + col < p.CG, gate = p.z != nullptr;
        auto has = [&](int t0, int r) { return row0 + r * RS < TT && t0 + row0 + r * RS < eos && cok; };
        auto copy_rows = [&](uint4(&to)[ST][TT][CH], const void* from, int64_t ld, int i) {
            const int t0 = bos + i * TT;
#pragma unroll
            for (int r = 0; r < NV; ++r) {
                const int64_t t = t0 + row0 + r * RS;
                if (has(t0, r)) copy16_async(&to[i % ST][row0 + r * RS][ch], static_cast<const T*>(from) + t * ld + c0 + col);
            }
        };
        if (first) {
            float2 bias[VN / 2];
#pragma unroll
            for (int e = 0; e < VN / 2; ++e)
                bias[e] = cok && p.bias ? make_float2(__ldg(p.bias + c0 + col + 2 * e), __ldg(p.bias + c0 + col + 2 * e + 1)) : both(0.f);
            auto copy = [&](int i) {
                copy_rows(sm.x, p.x, p.ldx, i);
                copy_rows(sm.dt, p.dt, p.lddt, i);
#pragma unroll
                for (int r = 0; r < NB; ++r) {
                    const int v = tid + F::SIDE * r, which = v / (TT * BCH), w = v % (TT * BCH);
                    const int64_t t = bos + i * TT + w / BCH;
                    const int e = g * S + (w % BCH) * VN;
                    if (which < 2 && t < eos)
                        copy16_async(&sm.bc[i % ST][v], which ? static_cast<const T*>(p.Cm) + t * p.ldC + e : static_cast<const T*>(p.B) + t * p.ldB + e);
                }
                copy_commit();
            };
            for (int i = 0; i < ST - 1; ++i) copy(i);
            for (int i = 0; i < tiles; ++i) {
                const int b2 = i & 1, b3 = i % ST;
                copy(i + ST - 1);
                copy_wait<ST - 1>();
                if (i >= 2) bar_sync(kFree + b2, kPair);
#pragma unroll
                for (int r = 0; r < NV; ++r) {
                    const int tt = row0 + r * RS;
                    if (tt < TT) {
                        float2 xv[VN / 2], dv[VN / 2];
                        unpack2(sm.x[b3][tt][ch], xv);
                        unpack2(sm.dt[b3][tt][ch], dv);
                        float4* to = reinterpret_cast<float4*>(&sm.d[b2][tt][col + (col / 16) * 2]);
#pragma unroll
                        for (int e = 0; e < VN / 2; ++e) {
                            const float2 d = step_of(dv[e], bias[e], p.softplus);
                            const float2 dx = __fmul2_rn(d, xv[e]);
                            to[e] = make_float4(d.x, dx.x, d.y, dx.y);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < NB; ++r) {
                    const int v = tid + F::SIDE * r, which = v / (TT * BCH), w = v % (TT * BCH);
                    if (which < 2) {
                        float f[VN];
                        unpack(sm.bc[b3][v], f);
#pragma unroll
                        for (int e = 0; e < VN; e += 4) {
                            const int q = ((w % BCH) * VN + e) / 4;
                            sm.b[b2][which][w / BCH][(q & 1) * L + q / 2] = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                        }
                    }
                }
                bar_arrive(kFull + b2, kPair);
            }
        } else {
            float2 D[VN / 2];
#pragma unroll
            for (int e = 0; e < VN / 2; ++e)
                D[e] = cok && p.D ? make_float2(__ldg(p.D + c0 + col + 2 * e), __ldg(p.D + c0 + col + 2 * e + 1)) : both(0.f);
            auto copy = [&](int i) {
                copy_rows(sm.x2, p.x, p.ldx, i);
                if (gate) copy_rows(sm.z, p.z, p.ldz, i);
                copy_commit();
            };
            for (int i = 0; i < ST - 1; ++i) copy(i);
            for (int i = 0; i < tiles; ++i) {
                const int b2 = i & 1, b3 = i % ST, t0 = bos + i * TT;
                copy(i + ST - 1);
                copy_wait<ST - 1>();
                bar_sync(kDone + b2, kPair);
#pragma unroll
                for (int r = 0; r < NV; ++r) {
                    const int tt = row0 + r * RS;
                    if (has(t0, r)) {
                        float2 xv[VN / 2], zv[VN / 2], sig;
                        float out[VN];
                        unpack2(sm.x2[b3][tt][ch], xv);
                        if (gate) unpack2(sm.z[b3][tt][ch], zv);
#pragma unroll
                        for (int e = 0; e < VN / 2; ++e) {
                            float2 o = *reinterpret_cast<const float2*>(&sm.y[b2][tt][0][col + 2 * e]);
                            if constexpr (F::UP > 1) o = __fadd2_rn(o, *reinterpret_cast<const float2*>(&sm.y[b2][tt][1][col + 2 * e]));
                            o = __ffma2_rn(D[e], xv[e], o);
                            if (gate) o = __fmul2_rn(o, silu2(zv[e], sig));
                            out[2 * e] = o.x, out[2 * e + 1] = o.y;
                        }
                        st16_stream(static_cast<T*>(p.y) + (int64_t)(t0 + tt) * p.C + c0 + col, pack(out));
                    }
                }
                if (i + 2 < tiles) bar_arrive(kLeft + b2, kPair);
            }
        }
        copy_wait<0>();
        return;
    }

    if constexpr (Q > 1) regs_more<kRegsWalk>();
    const int j = threadIdx.x % L, cl = threadIdx.x / L * Q;
    const bool ok = cg0 + cl < p.CG;  // all Q or none: p.CG is a multiple of 8
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    const bool has_slot = slot >= 0 && slot < p.num_slots;
    const bool use_init = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0);
    const int64_t own = ok ? (int64_t)(c0 + cl) * S + 8 * j : 0;
    float* st = p.state + (int64_t)slot * p.C * S + own;
    float2 A2[Q][4], h[Q][4];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = (ok ? q * S : 0) + 4 * i;
            float2 t[2];
            load4(p.A_log + own + at, t);
            A2[q][2 * i] = make_float2(a_log2(t[0].x), a_log2(t[0].y)), A2[q][2 * i + 1] = make_float2(a_log2(t[1].x), a_log2(t[1].y));
            const float4 u = use_init ? *reinterpret_cast<const float4*>(st + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[q][2 * i] = make_float2(u.x, u.y), h[q][2 * i + 1] = make_float2(u.z, u.w);
        }
    for (int i = 0; i < tiles; ++i) {
        const int b2 = i & 1, len = min(TT, eos - bos - i * TT);
        bar_sync(kFull + b2, kPair);
        if (i >= 2) bar_sync(kLeft + b2, kPair);
        auto token = [&](int tt, float (&sum)[Q]) {  // one token on; this lane's 8 states' sums
            float2 d[Q], acc[Q];
            if constexpr (Q == 2) {
                const float4 v = *reinterpret_cast<const float4*>(&sm.d[b2][tt][cl + (cl / 16) * 2]);
                d[0] = make_float2(v.x, v.y), d[1] = make_float2(v.z, v.w);
            } else {
                d[0] = sm.d[b2][tt][cl + (cl / 16) * 2];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 b = sm.b[b2][0][tt][k * L + j], c = sm.b[b2][1][tt][k * L + j];
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    advance(h[q][2 * k], A2[q][2 * k], both(d[q].x), both(d[q].y), make_float2(b.x, b.y));
                    advance(h[q][2 * k + 1], A2[q][2 * k + 1], both(d[q].x), both(d[q].y), make_float2(b.z, b.w));
                    acc[q] = k ? __ffma2_rn(h[q][2 * k], make_float2(c.x, c.y), acc[q]) : __fmul2_rn(h[q][0], make_float2(c.x, c.y));
                    acc[q] = __ffma2_rn(h[q][2 * k + 1], make_float2(c.z, c.w), acc[q]);
                }
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) sum[q] = __fadd_rn(acc[q].x, acc[q].y);
        };
        constexpr int LP = L / F::UP;  // lanes of a part
        auto put = [&](int tt, const float (&v)[Q]) {
            if constexpr (Q == 2) *reinterpret_cast<float2*>(&sm.y[b2][tt][j / LP][cl]) = make_float2(v[0], v[1]);
            else sm.y[b2][tt][0][cl] = v[0];
        };
        constexpr int U = TT;  // tokens whose loads and exponentials run ahead of the recurrence (Q = 1: 564 us for the 16 prompts, 8 of them 578)
        if (len == TT) {
#pragma unroll 1
            for (int tt = 0; tt < TT; tt += U) {
                float s[U][Q];
#pragma unroll
                for (int k = 0; k < U; ++k) token(tt + k, s[k]);
#pragma unroll
                for (int k = 0; k < U; k += LP) {
                    float v[Q];
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        float g[LP];
#pragma unroll
                        for (int e = 0; e < LP; ++e) g[e] = s[k + e][q];
                        v[q] = scatter_sum<LP>(g, j % LP);
                    }
                    put(tt + k + j % LP, v);
                }
            }
        } else {
            for (int tt = 0; tt < len; ++tt) {
                float s[Q];
                token(tt, s);
#pragma unroll
                for (int q = 0; q < Q; ++q)
#pragma unroll
                    for (int off = 1; off < LP; off <<= 1) s[q] = __fadd_rn(s[q], __shfl_xor_sync(0xffffffffu, s[q], off));
                if (j % LP == 0) put(tt, s);
            }
        }
        if (i + 2 < tiles) bar_arrive(kFree + b2, kPair);
        bar_arrive(kDone + b2, kPair);
    }
    if (has_slot && ok) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float4*>(st + q * S + 4 * i) = make_float4(h[q][2 * i].x, h[q][2 * i].y, h[q][2 * i + 1].x, h[q][2 * i + 1].y);
    }
}

// Single tokens: HBM bound by the states, read and written once.  A lane holds 4 states (16 bytes)
// of a channel, L = S / 4 lanes a channel, a CTA 128 / L channels of `rows` batch rows, whose A and
// D it reads once and whose B and C it keeps in shared memory in fp32.  RW rows go together: lane
// j does the work per (row, channel) of row j, softplus before and skip, gate and store after, so
// that no lane repeats it, and the rows' states are in flight at once.  (Loading the next rows ahead
// costs registers and with them CTAs: 53 us instead of 51 for 256 x 8192 x 16.)
constexpr int kUpdRows = 16;

template <typename T, int S>
__global__ void __launch_bounds__(128) scan_update_kernel(const __grid_constant__ Params p, int rows) {
    constexpr int L = S / 4, CB = 128 / L, RW = L < 4 ? L : 4;
    constexpr uint32_t all = 0xffffffffu;
    __shared__ float4 bc[kUpdRows][2][S / 4];
    const int nb = p.bpg * p.G, blk = blockIdx.x % nb, b0 = blockIdx.x / nb * rows, nr = min(rows, p.N - b0);
    const int g = blk / p.bpg, j = threadIdx.x % L, jr = j % RW;
    const int cg = (blk % p.bpg) * CB + threadIdx.x / L;
    const bool ok = cg < p.CG;
    const int c = g * p.CG + (ok ? cg : 0);
    float* st = p.state + (int64_t)c * S + 4 * j;
    const int64_t CS = (int64_t)p.C * S;
    float2 h[RW][2];
    int slot[RW];
    float x, dt, z;
    auto load = [&](int r0) {
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int row = b0 + r0 + r;
            slot[r] = r0 + r < nr ? (p.idx ? __ldg(p.idx + row) : row) : -1;
            if (slot[r] >= p.num_slots) slot[r] = -1;
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const float4 s = slot[r] >= 0 ? *reinterpret_cast<const float4*>(st + slot[r] * CS) : make_float4(0.f, 0.f, 0.f, 0.f);
            h[r][0] = make_float2(s.x, s.y), h[r][1] = make_float2(s.z, s.w);
        }
        const int64_t row = b0 + min(r0 + jr, nr - 1);
        x = load1(static_cast<const T*>(p.x) + row * p.ldx + c);
        dt = load1(static_cast<const T*>(p.dt) + row * p.lddt + c);
        z = p.z ? load1(static_cast<const T*>(p.z) + row * p.ldz + c) : 0.f;
    };
    load(0);
    for (int i = threadIdx.x; i < nr * (S / 2); i += 128) {
        const int r = i / (S / 2), which = i % (S / 2) / (S / 4), q = i % (S / 4);
        const int64_t row = b0 + r;
        float2 v[2];
        load4((which ? static_cast<const T*>(p.Cm) + row * p.ldC : static_cast<const T*>(p.B) + row * p.ldB) + (int64_t)g * S + 4 * q, v);
        bc[r][which][q] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
    float2 A2[2];
    load4(p.A_log + (int64_t)c * S + 4 * j, A2);
    A2[0] = make_float2(a_log2(A2[0].x), a_log2(A2[0].y)), A2[1] = make_float2(a_log2(A2[1].x), a_log2(A2[1].y));
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f, D = p.D ? __ldg(p.D + c) : 0.f;
    __syncthreads();
    for (int r0 = 0; r0 < nr; r0 += RW) {
        if (r0) load(r0);
        const float d = step_of(both(dt), both(bias), p.softplus).x, dx = __fmul_rn(d, x);
        float mine = 0.f;
        int mine_slot = -1;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int at = min(r0 + r, nr - 1), from = (threadIdx.x & 31 & ~(L - 1)) + r;
            const float dr = __shfl_sync(all, d, from), dxr = __shfl_sync(all, dx, from);
            const float4 b = bc[at][0][j], k = bc[at][1][j];
            const float2 cc[2] = {make_float2(k.x, k.y), make_float2(k.z, k.w)};
            advance(h[r][0], A2[0], both(dr), both(dxr), make_float2(b.x, b.y));
            advance(h[r][1], A2[1], both(dr), both(dxr), make_float2(b.z, b.w));
            const float t = __shfl_sync(all, sum_states4<L>(h[r], cc, j), (threadIdx.x & 31 & ~(L - 1)) + 1);
            if (jr == r) mine = t, mine_slot = slot[r];
            if (ok && slot[r] >= 0)
                *reinterpret_cast<float4*>(st + slot[r] * CS) = make_float4(h[r][0].x, h[r][0].y, h[r][1].x, h[r][1].y);
        }
        float y = __fmaf_rn(D, x, mine);
        float2 sig;
        if (p.z) y = __fmul_rn(y, silu2(both(z), sig).x);
        if (ok && j < RW && mine_slot >= 0) store1(static_cast<T*>(p.y) + (int64_t)(b0 + r0 + j) * p.C + c, y);
    }
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

// K<T, S>::go launches over p.N sequences (rows) and the channel blocks; K<T, S>::cb: channels of a CTA.
template <template <typename, int> class K, typename T, int S>
gdn_status launch(cudaStream_t s, Params& p) {
    constexpr int cb = K<T, S>::cb;
    p.bpg = (p.CG + cb - 1) / cb;
    if ((long long)p.N * p.G * p.bpg >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
    return K<T, S>::go((unsigned)(p.G * p.bpg), s, p);
}
template <template <typename, int> class K, typename T>
gdn_status by_states(int S, cudaStream_t s, Params& p) {
    switch (S) {
        case 8: return launch<K, T, 8>(s, p);
        case 16: return launch<K, T, 16>(s, p);
        case 32: return launch<K, T, 32>(s, p);
        case 64: return launch<K, T, 64>(s, p);
    }
    return GDN_ERR_UNSUPPORTED;
}
template <typename T, int S>
struct FwdK {
    static constexpr int cb = FwdTile<T, S, 1>::CB;
    template <int Q>
    static gdn_status run(cudaStream_t s, const Params& p) {
        using F = FwdTile<T, S, Q>;
        if (cudaFuncSetAttribute(scan_fwd_kernel<T, S, Q>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess)
            return GDN_ERR_CUDA;
        Params q = p;
        q.bpg = (p.CG + F::CB - 1) / F::CB;
        const unsigned blocks = (unsigned)(q.bpg * q.G);
        const long long n = p.N;
        q.ranked = n > 1 && n <= kRanked && blocks * n > kSMs && n * n * n <= 256LL * p.T;
        scan_fwd_kernel<T, S, Q><<<blocks * p.N, F::NT, sizeof(F), s>>>(q);
        return launch_status();
    }
    static gdn_status go(unsigned blocks, cudaStream_t s, const Params& p) {
        // Two channels a lane from more than the three blocks on that an SM holds at once (4096 tokens x
        // 8192 x 64, 3.4 blocks an SM: 913 and 581 us; with fewer, figures above, they leave SMs idle).  The
        // longest of N sequences is taken for up to min(N, 3) mean lengths: once it walks alone, a token
        // takes twice as long with two channels a lane (16 ragged prompts, 12265 x 2760 x 16, 4.6 blocks an
        // SM: 192 and 343 us; 16384 x 8192 x 16, 13 blocks: 564 and 536).  Not for 8 states: their walkers
        // would be half a warpgroup.  The bits are the same either way, so a compiler that leaves too few
        // registers to move costs time only.
        if constexpr (S >= 16) {
            static std::atomic<int> known{0};
            if ((long long)blocks * p.N > 3LL * kSMs * (p.N < 3 ? p.N : 3)) {
                const gdn_status st = check_registers(scan_fwd_kernel<T, S, 2>, FwdTile<T, S, 2>::NT, 128 * (kRegsSide + kRegsWalk), known);
                if (st != GDN_ERR_UNSUPPORTED) return st == GDN_OK ? run<2>(s, p) : st;
            }
        }
        return run<1>(s, p);
    }
};
template <typename T, int S>
struct UpdK {
    static constexpr int cb = 128 / (S / 4);
    // Many rows a CTA where that leaves every SM several CTAs; else as few as go together.
    static gdn_status go(unsigned blocks, cudaStream_t s, const Params& p) {
        const int most = (int)((long long)blocks * p.N / (kSMs * 16));
        const int rows = most >= kUpdRows ? kUpdRows : most >= 8 ? 8 : 4;
        scan_update_kernel<T, S><<<blocks * ((p.N + rows - 1) / rows), 128, 0, s>>>(p, rows);
        return launch_status();
    }
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
