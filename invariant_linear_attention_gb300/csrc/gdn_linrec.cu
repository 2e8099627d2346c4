// gdn_linrec.cu -- the gated linear recurrence: prompts (and the trainer's forward), single tokens and
// the gradient.  The arithmetic is in gdn_linrec.cuh.
#include <type_traits>

#include "gdn_async.cuh"
#include "gdn_host.h"
#include "gdn_linrec.cuh"

namespace gdn {
namespace {

using namespace linrec;

// Prompts.  A CTA walks one sequence over CB channels in tiles of TT tokens.  Nearly all the work of a token does not
// depend on the one before it: only h <- a h + b does, 5 cycles a token.  So
//   * the workers, each four tokens of two channels (fp32: of one), in step i finish tile i - NB (gate, stores of y) and prepare
//     tile i (a and b, to shared memory);
//   * the walkers, a lane a channel, walk tile after tile and leave h in b's place.
// A worker reads the h of the very places that it then writes, so it meets nobody but the walkers, NB tiles behind or ahead:
// at named barriers full (a tile prepared) and done (it is walked), one of each per buffer, which every side passes once a
// tile.  The inputs arrive by asynchronous 16-byte copies, AHEAD tiles ahead, for a group of workers that copies what it reads.
//
// What bounds it.  fp32: HBM (16 prompts, 32768 x 4096, gated: 398 us, 0.99 of the measured peak).  bf16 with full SMs (16
// prompts, 32768 x 4096, gated: 264 us, 0.75): nothing alone; issue slots are half taken, the special function units (72
// cycles for 256 values; 160 us by themselves before the gates shared a reciprocal) and the path from shared memory as well,
// by 18 warps an SM that the registers and 108 KB of buffers leave.  (When it took 284 us: 240 with trivial work in the workers'
// place, 261 without the walk.)  A single sequence: the walk, 6.0 ns a token with its stores and the workers beside it (65536 x 2048:
// 396 us; the workers without it 300), 3.7 ns alone; its dependent steps by themselves 2.6 ns.
template <typename T, int CB, int WORKERS>
struct FwdTile {
    static constexpr int VN = V16<T>::n, CH = CB / VN, WORK = WORKERS, TT = WORK / CH, WALK = CB < 32 ? 32 : CB, NT = WORK + WALK;
    static constexpr int AHEAD = 2, ST = AHEAD + 1, NB = 3;
    static constexpr int GROUP = VN == 8 && CB == 32 ? 64 : 32;     // threads that copy for one another
    static constexpr int kFull = 1, kDone = kFull + NB, kGroup = kDone + NB;  // barriers
    // Four tokens of a channel are 16 bytes, the walker's unit (with 4-byte loads its three a token took 14 cycles, not 5).
    // Unit q of channel c lies at unit(q, c) of its row: eight neighbouring lanes of a worker warp, two channels of four
    // rows, then meet no bank twice.
    float4 a[NB][TT / 4][CB], b[NB][TT / 4][CB];
    static __device__ __forceinline__ int unit(int q, int c) { return c ^ 2 * (q & 3); }
    uint4 in[ST][4][WORK];                                    // x, a_gate, x_gate of a tile, z of the one NB before
    uint4 out[NB][std::is_same<T, float>::value ? 1 : WORK];  // bf16: y on its way from columns to rows; a group of two warps stores it a step later
    float K[CB];
    static_assert(ST == 3 && NB == 3, "a step's copies and buffers come round together");
    static_assert(CB <= 32 && TT % 16 == 0, "rows of at most 128 bytes, tiles of whole walks");
    static_assert(kGroup + (GROUP > 32 ? WORK / GROUP : 0) <= 16, "barriers of a CTA");
};

__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// A worker's share of a tile: tokens 4 q .. 4 q + 3 of its channels.  v: packed pairs of tokens, those of one channel and then,
// in bf16, those of the other.
template <typename T, int CB>
struct Share;

// bf16: a warp takes 16 tokens of 16 channels, lane l channels l / 4 and l / 4 + 8 and tokens 4 (l % 4) ..  Four 8 x 8 matrices, two
// of tokens 0, 1, 4, 5, .. and two of tokens 2, 3, 6, 7, .., each transposed on the way from and to the rows in memory,
// put two tokens of a channel into one register: 1 instruction an input where loads of a row's pairs took 4.
template <int CB>
struct Share<__nv_bfloat16, CB> {
    static constexpr int NP = 4, CH = CB / 8;
    int c, q, at;  // c: within the CTA's channels; at: byte offset of this lane's matrix row in an input
    // The 16-byte place of chunk ch of row t: a matrix's eight rows (above) lie in eight different places of a 128-byte line.
    static __device__ __forceinline__ int place(int t, int ch, int chunks) {
        const int g = (t >> 2) & 3;
        return chunks == 4 ? t * 4 + (ch ^ g) : ((t * 2 + ch) & ~7) | (((t * 2 + ch) & 7) ^ ((g & 1) | (g & 2) << 1));
    }
    __device__ __forceinline__ Share(int tid) {
        const int l = tid % 32, w = tid / 32, cw = w % (CB / 16), tb = w / (CB / 16) * 16;
        const int r = l % 8, t = (r >> 1) * 4 + (r & 1) + (l & 8 ? 2 : 0);
        c = cw * 16 + l / 4, q = tb / 4 + l % 4;
        at = 16 * place(tb + t, cw * 2 + l / 16, CH);
    }
    __device__ __forceinline__ int first() const { return q & ~3; }  // its warp's first unit
    __device__ __forceinline__ void rates(const float* K, float2 (&k)[4]) const { k[0] = k[1] = both(K[c]), k[2] = k[3] = both(K[c + 8]); }
    __device__ __forceinline__ void load(const uint4* in, float2 (&v)[4]) const {
        uint32_t u[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                     : "r"(smem_u32(in) + at)
                     : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = make_float2(bf_lo(u[j]), bf_hi(u[j]));
    }
    template <typename F>
    __device__ __forceinline__ void put(float4 (*to)[CB], const float2 (&v)[4]) const {
        to[q][F::unit(q, c)] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y), to[q][F::unit(q, c + 8)] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
    template <typename F>
    __device__ __forceinline__ void get(const float4 (*from)[CB], float2 (&v)[4]) const {
        const float4 x = from[q][F::unit(q, c)], y = from[q][F::unit(q, c + 8)];
        v[0] = make_float2(x.x, x.y), v[1] = make_float2(x.z, x.w), v[2] = make_float2(y.x, y.y), v[3] = make_float2(y.z, y.w);
    }
    static __device__ __forceinline__ void transposed(uint32_t to, const float2 (&v)[4]) {
        const uint32_t u[4] = {bf_pack(v[0].x, v[0].y), bf_pack(v[1].x, v[1].y), bf_pack(v[2].x, v[2].y), bf_pack(v[3].x, v[3].y)};
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
    }
    // To the places that its warp read an input from.
    __device__ __forceinline__ void put_in(uint4* in, const float2 (&v)[4]) const { transposed(smem_u32(in) + at, v); }
};
// fp32: a lane one channel; a warp's lanes are neighbouring channels.
template <int CB>
struct Share<float, CB> {
    static constexpr int NP = 2, CH = CB / 4;
    int c, q;
    // Rows of 64 bytes share a line, in an order that goes by the row's unit too: a warp reads one row of each of two units.
    static __device__ __forceinline__ int place(int t, int ch, int chunks) { return (chunks == 8 ? t : (t & ~1) | ((t ^ (t >> 2)) & 1)) * chunks + ch; }
    __device__ __forceinline__ Share(int tid) { c = tid % CB, q = tid / CB; }
    __device__ __forceinline__ int first() const { return q; }
    __device__ __forceinline__ void rates(const float* K, float2 (&k)[2]) const { k[0] = k[1] = both(K[c]); }
    __device__ __forceinline__ void load(const uint4* in, float2 (&v)[2]) const {
        const float* f = reinterpret_cast<const float*>(in);
        auto at = [&](int j) { return f[4 * place(4 * q + j, c / 4, CH) + c % 4]; };
        v[0] = make_float2(at(0), at(1)), v[1] = make_float2(at(2), at(3));
    }
    template <typename F>
    __device__ __forceinline__ void put(float4 (*to)[CB], const float2 (&v)[2]) const {
        to[q][F::unit(q, c)] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
    template <typename F>
    __device__ __forceinline__ void get(const float4 (*from)[CB], float2 (&v)[2]) const {
        const float4 x = from[q][F::unit(q, c)];
        v[0] = make_float2(x.x, x.y), v[1] = make_float2(x.z, x.w);
    }
};

// The sequence of rank `rank` by length, the longest first (ties by number), so that the longest walks do not start last.
// A CTA's N^2 comparisons have to be few against its walk of T / N tokens: up to N^3 = 256 T, as for the selective scan.
constexpr int kRanked = 256;
__device__ __forceinline__ int ranked(const Params& p, int rank, int threads) {
    __shared__ int lens[kRanked], found;
    for (int i = threadIdx.x; i < p.N; i += threads) {
        int bos, eos;
        bounds(p.cu, i, p.T, bos, eos);
        lens[i] = eos - bos;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.N; i += threads) {
        const int mine = lens[i];
        int before = 0;
        for (int k = 0; k < p.N; ++k) before += lens[k] > mine || (lens[k] == mine && k < i);
        if (before == rank) found = i;
    }
    __syncthreads();
    return found;
}

// Sequence n over the CTA's channels.
template <typename T, typename F, int CB, Kind KIND>
__device__ __forceinline__ void walk_sequence(const Params& p, F& sm, int n, int c0) {
    using Q = Share<T, CB>;
    constexpr int VN = F::VN, NP = Q::NP, CH = F::CH, TT = F::TT, WORK = F::WORK, AHEAD = F::AHEAD, ST = F::ST;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int len = eos - bos, tiles = (len + TT - 1) / TT;
    if (threadIdx.x >= F::WALK) {
        const int tid = threadIdx.x - F::WALK;
        const bool gate = p.z != nullptr;
        // its copies: a chunk of row tid / CH of each tile
        const int row = tid / CH, slot = Q::place(row, tid % CH, CH), cc = c0 + tid % CH * VN;
        const int upto = cc < p.C ? max(len - row, 0) : 0;  // tiles that start before this token have a row to copy
        auto at = [&](const void* from, int64_t ld, int t) { return static_cast<const char*>(from) + ((int64_t)(bos + row + t) * ld + cc) * (int64_t)sizeof(T); };
        const char *px = at(p.x, p.ldx, 0), *pa = at(p.ag, p.lda, 0), *pg = at(p.xg, p.ldg, 0), *pz = at(p.z, p.ldz, -F::NB * TT);
        auto copy = [&](int stage, int t) {  // what the step whose tile starts at t needs
            uint4(&to)[4][WORK] = sm.in[stage];
            if (t < upto) {
                copy16_async(&to[0][slot], px);
                copy16_async(&to[1][slot], pa);
                if (has_gate<KIND>(p)) copy16_async(&to[2][slot], pg);
            }
            if (gate && (unsigned)(t - F::NB * TT) < (unsigned)upto) copy16_async(&to[3][slot], pz);
            px += p.sx, pa += p.sa, pg += p.sg, pz += p.sz;
            copy_commit();
        };
        const Q my(tid);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) copy(i, i * TT);
        float2 K[NP];
        my.rates(sm.K, K);
        const bool far = any_far(K);
        constexpr bool bf16 = !std::is_same<T, float>::value, later = bf16 && F::GROUP > 32;
        const int mine = 4 * my.first();  // its warp's first token of a tile
        char* y = static_cast<char*>(p.y) + (bf16 ? (int64_t)(bos + row) * p.C + cc : (int64_t)(bos + 4 * my.q) * p.C + c0 + my.c) * (int64_t)sizeof(T);
        // Step i, J = i % 3: the tile from token t on, and the one NB before.
        auto step = [&](auto J_, int i, int t) {
            constexpr int J = decltype(J_)::value, before = (J + 2) % 3;
            copy_wait<AHEAD - 1>();
            if (F::GROUP > 32) bar_sync(F::kGroup + tid / F::GROUP, F::GROUP);
            else __syncwarp();
            copy((J + AHEAD) % ST, t + AHEAD * TT);
            const uint4(&from)[4][WORK] = sm.in[J];
            auto flush = [&](int which, int old) {  // bf16: a row of the tile from `old` on
                if (old < upto) st16_stream(y, sm.out[which][slot]);
                y += p.sy;
            };
            const int old = t - F::NB * TT;
            if (later && i > F::NB) flush(before, old - TT);
            if (i >= F::NB && i < tiles + F::NB) {
                bar_sync(F::kDone + J, F::NT);
                if (old + mine < len) {
                    float2 h[NP];
                    my.template get<F>(sm.b[J], h);
                    if (gate) {
                        float2 z[NP];
                        my.load(from[3], z);
                        branch(p.act, z, h);
                    }
                    if constexpr (bf16) {
                        if (!later) __syncwarp();
                        my.put_in(sm.out[J], h);
                        if (!later) {
                            __syncwarp();
                            flush(J, old);
                        }
                    } else {
                        const float f[4] = {h[0].x, h[0].y, h[1].x, h[1].y};
                        const int has = c0 + my.c < p.C ? len - old - mine : 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < has) __stcs(reinterpret_cast<float*>(y) + (int64_t)j * p.C, f[j]);
                        y += p.sy;
                    }
                }
            }
            if (i < tiles) {
                if (t + mine < len) {
                    float2 x[NP], ag[NP], xg[NP], a[NP], b[NP];
                    my.load(from[0], x);
                    my.load(from[1], ag);
                    my.load(from[2], xg);
                    steps<KIND>(p, far, K, ag, xg, x, a, b);
                    my.template put<F>(sm.a[J], a);
                    my.template put<F>(sm.b[J], b);
                }
                bar_arrive(F::kFull + J, F::NT);
            }
        };
        const int last = tiles + F::NB + later;
        for (int i = 0, t = 0; i < last; i += 3, t += 3 * TT) {
            step(std::integral_constant<int, 0>{}, i, t);
            if (i + 1 < last) step(std::integral_constant<int, 1>{}, i + 1, t + TT);
            if (i + 2 < last) step(std::integral_constant<int, 2>{}, i + 2, t + 2 * TT);
        }
        copy_wait<0>();
        return;
    }

    const int cl = threadIdx.x % CB, c = c0 + cl;
    const bool walks = CB == F::WALK || threadIdx.x < CB;  // with 16 channels the other half of the warp passes the barriers only
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    const bool has_slot = walks && c < p.C && slot >= 0 && slot < p.num_slots;
    float* st = p.state + (int64_t)slot * p.C + c;
    float h = has_slot && (!p.has_init || __ldg(p.has_init + n) != 0) ? *st : 0.f;
    for (int i = 0, buf = 0; i < tiles; ++i) {
        const int here = walks ? min(TT, len - i * TT) : 0;
        bar_sync(F::kFull + buf, F::NT);
        // S sets of V units in registers: while one is walked, the loads of the others are under way (at the end they read on
        // into what follows, unused).
        constexpr int S = 2, V = 4;
        const int units = here / 4;
        float4 (*pa)[CB] = sm.a[buf], (*pb)[CB] = sm.b[buf];
        int u = 0;
        auto walk4 = [&](const float4& av, const float4& bv) {
            float4 o;
            h = o.x = __fmaf_rn(av.x, h, bv.x), h = o.y = __fmaf_rn(av.y, h, bv.y), h = o.z = __fmaf_rn(av.z, h, bv.z), h = o.w = __fmaf_rn(av.w, h, bv.w);
            return o;
        };
        if (units >= S * V) {
            const float4* ra[4];  // units 0 to 3, and every fourth from there
            float4* rb[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) ra[k] = &pa[0][F::unit(k, cl)], rb[k] = &pb[0][F::unit(k, cl)];
            float4 ak[S][V], bk[S][V];
            auto load = [&](int unit, int set) {  // from this turn's first unit on
#pragma unroll
                for (int k = 0; k < V; ++k) ak[set][k] = ra[(unit + k) & 3][(unit + k) * CB], bk[set][k] = rb[(unit + k) & 3][(unit + k) * CB];
            };
#pragma unroll
            for (int j = 0; j < S - 1; ++j) load(j * V, j);
            for (; u + S * V <= units; u += S * V) {
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    load((j + S - 1) * V, (j + S - 1) % S);
#pragma unroll
                    for (int k = 0; k < V; ++k) rb[(j * V + k) & 3][(j * V + k) * CB] = walk4(ak[j][k], bk[j][k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) ra[k] += S * V * CB, rb[k] += S * V * CB;
            }
        }
        for (; 4 * u < here; ++u) {
            const float4 av = pa[u][F::unit(u, cl)], bv = pb[u][F::unit(u, cl)];
            if (u < units) {
                pb[u][F::unit(u, cl)] = walk4(av, bv);
            } else {
                const float af[3] = {av.x, av.y, av.z}, bf[3] = {bv.x, bv.y, bv.z};
                float o[3] = {0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (4 * u + k < here) h = o[k] = __fmaf_rn(af[k], h, bf[k]);
                pb[u][F::unit(u, cl)] = make_float4(o[0], o[1], o[2], 0.f);
            }
        }
        if (CB != F::WALK) __syncwarp();
        bar_arrive(F::kDone + buf, F::NT);
        buf = buf + 1 == F::NB ? 0 : buf + 1;
    }
    if (has_slot) *st = h;
}

template <typename F, int CB, Kind KIND>
__device__ __forceinline__ void load_rates(const Params& p, F& sm, int c0) {
    if (has_param<KIND>(p) && threadIdx.x < CB) sm.K[threadIdx.x] = c0 + (int)threadIdx.x < p.C ? rate_of(__ldg(p.ap + c0 + threadIdx.x), p.decay) : 0.f;
    __syncthreads();
}

template <typename T, typename F, int CB, int CTAS, Kind KIND>
__global__ void __launch_bounds__(F::NT, CTAS) linrec_fwd_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const int blocks = (p.C + CB - 1) / CB, order = blockIdx.x / blocks, c0 = blockIdx.x % blocks * CB;
    const int n = p.ranked ? ranked(p, order, F::NT) : order;
    load_rates<F, CB, KIND>(p, sm, c0);
    walk_sequence<T, F, CB, KIND>(p, sm, n, c0);
}

// Many sequences, most of them short: a CTA for each would cost 2.3 us whatever it holds.  Those of up to kShort tokens go to
// linrec_short_kernel, a thread a chunk of channels of a sequence; here a CTA takes all the longer ones among sequences g, g + groups, ..
constexpr int kShort = 32;
template <typename T, typename F, int CB, int CTAS, Kind KIND>
__global__ void __launch_bounds__(F::NT, CTAS) linrec_long_kernel(const __grid_constant__ Params p, int groups) {
    extern __shared__ __align__(128) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const int blocks = (p.C + CB - 1) / CB, g = blockIdx.x / blocks, c0 = blockIdx.x % blocks * CB;
    bool first = true;
    for (int64_t base = g; base < p.N; base += 32 * groups) {  // every warp looks at the same 32 sequences
        const int64_t at = base + (int64_t)(threadIdx.x & 31) * groups;
        int bos = 0, eos = 0;
        if (at < p.N) bounds(p.cu, (int)at, p.T, bos, eos);
        for (unsigned longer = __ballot_sync(0xffffffffu, eos - bos > kShort); longer; longer &= longer - 1) {
            if (first) load_rates<F, CB, KIND>(p, sm, c0);
            else __syncthreads();  // the sequence before is through with the buffers
            first = false;
            walk_sequence<T, F, CB, KIND>(p, sm, (int)base + (__ffs(longer) - 1) * groups, c0);
        }
    }
}
// A chain of loads (place, slot, state), then a step a token, the next one's loads under way: 4096 sequences of 1 token x 4096, bf16: 0.40 of HBM.
template <typename T>
__global__ void __launch_bounds__(128) linrec_short_kernel(const __grid_constant__ Params p) {
    constexpr int VN = V16<T>::n, NP = VN / 2;
    const int chunks = p.C / VN, blocks = (chunks + 127) / 128, ch = blockIdx.x % blocks * 128 + threadIdx.x, c = ch * VN, n = blockIdx.x / blocks;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    if (ch >= chunks || eos - bos > kShort) return;
    const int slot = !p.state ? -1 : (p.idx ? __ldg(p.idx + n) : n);
    float4* st = slot >= 0 && slot < p.num_slots ? reinterpret_cast<float4*>(p.state + (int64_t)slot * p.C + c) : nullptr;
    const bool init = st && (!p.has_init || __ldg(p.has_init + n) != 0);
    struct Token {
        uint4 x, ag, xg, z;
    };
    auto load = [&](int64_t t) {
        Token k;
        k.xg = k.z = make_uint4(0u, 0u, 0u, 0u);
        k.x = ld16(static_cast<const T*>(p.x) + t * p.ldx + c), k.ag = ld16(static_cast<const T*>(p.ag) + t * p.lda + c);
        if (p.xg) k.xg = ld16(static_cast<const T*>(p.xg) + t * p.ldg + c);
        if (p.z) k.z = ld16(static_cast<const T*>(p.z) + t * p.ldz + c);
        return k;
    };
    Token next{};
    if (bos < eos) next = load(bos);
    float2 h[NP], K[NP];
#pragma unroll
    for (int e = 0; e < NP; e += 2) {
        const float4 v = init ? st[e / 2] : make_float4(0.f, 0.f, 0.f, 0.f);
        h[e] = make_float2(v.x, v.y), h[e + 1] = make_float2(v.z, v.w);
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) K[e] = p.ap ? make_float2(rate_of(__ldg(p.ap + c + 2 * e), p.decay), rate_of(__ldg(p.ap + c + 2 * e + 1), p.decay)) : both(0.f);
    const bool far = any_far(K);
#pragma unroll 1
    for (int t = bos; t < eos; ++t) {
        const Token k = next;
        if (t + 1 < eos) next = load(t + 1);
        float2 x[NP], ag[NP], xg[NP], a[NP], b[NP];
        unpack2(k.x, x);
        unpack2(k.ag, ag);
        unpack2(k.xg, xg);
        steps<kAny>(p, far, K, ag, xg, x, a, b);
#pragma unroll
        for (int e = 0; e < NP; ++e) x[e] = h[e] = __ffma2_rn(a[e], h[e], b[e]);
        if (p.z) {
            float2 z[NP];
            unpack2(k.z, z);
            branch(p.act, z, x);
        }
        st16(static_cast<T*>(p.y) + (int64_t)t * p.C + c, pack2(x));
    }
    if (!st) return;
#pragma unroll
    for (int e = 0; e < NP; e += 2) st[e / 2] = make_float4(h[e].x, h[e].y, h[e + 1].x, h[e + 1].y);
}

// Single tokens: a thread takes a chunk of channels over `rows` batch rows, so that it works out their rates once.  A launch and a chain
// of loads (slot, state) for small batches; 256 x 4096, bf16, gated: 6.4 us, 0.43 of HBM; 512 x 8192: 16.5 us, 0.68; 2048 x 8192: 52.9 us, 0.84 (fp32 68, 1.0).
template <typename T>
__global__ void __launch_bounds__(128) linrec_update_kernel(const __grid_constant__ Params p, int rows) {
    constexpr int VN = V16<T>::n, NP = VN / 2;
    const int chunks = p.C / VN, blocks = (chunks + 127) / 128, ch = blockIdx.x % blocks * 128 + threadIdx.x, c = ch * VN;
    if (ch >= chunks) return;
    const int first = blockIdx.x / blocks * rows, last = min(first + rows, p.N);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    float2 K[NP];
    bool far = false;
    for (int64_t n = first; n < last; ++n) {
        // A row's inputs do not wait for its slot, nor its loads for the rates.
        const int slot = p.idx ? __ldg(p.idx + n) : (int)n;
        const uint4 xr = ld16(static_cast<const T*>(p.x) + n * p.ldx + c), ar = ld16(static_cast<const T*>(p.ag) + n * p.lda + c);
        const uint4 gr = p.xg ? ld16(static_cast<const T*>(p.xg) + n * p.ldg + c) : none, zr = p.z ? ld16(static_cast<const T*>(p.z) + n * p.ldz + c) : none;
        const bool live = slot >= 0 && slot < p.num_slots;
        float4* st = reinterpret_cast<float4*>(p.state + (int64_t)(live ? slot : 0) * p.C + c);
        float4 v[NP / 2];
#pragma unroll
        for (int e = 0; e < NP / 2; ++e) v[e] = live ? st[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        if (n == first) {
#pragma unroll
            for (int e = 0; e < NP; ++e) K[e] = p.ap ? make_float2(rate_of(__ldg(p.ap + c + 2 * e), p.decay), rate_of(__ldg(p.ap + c + 2 * e + 1), p.decay)) : both(0.f);
            far = any_far(K);
        }
        if (!live) continue;
        float2 h[NP], x[NP], ag[NP], xg[NP], a[NP], b[NP];
#pragma unroll
        for (int e = 0; e < NP; e += 2) h[e] = make_float2(v[e / 2].x, v[e / 2].y), h[e + 1] = make_float2(v[e / 2].z, v[e / 2].w);
        unpack2(xr, x);
        unpack2(ar, ag);
        unpack2(gr, xg);
        steps<kAny>(p, far, K, ag, xg, x, a, b);
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

// Gradient.  A tile is TT tokens of one sequence (its last one may be shorter); what reaches it from the tokens before
// and behind is linear in two numbers a channel, so tiles run side by side:
//   linrec_sum_kernel: of each tile the product P of its decays, its last state from 0 and the gradient that leaves it backwards with 0 from behind
//   linrec_join_kernel: a sequence's tiles in order, H <- P H + h, and in reverse, G <- P G + g: the state before each tile, the gradient from behind it
//   linrec_bwd_kernel: each tile again from these, with its gradients
// With e = dy act(z) and G_t = e_t + a_{t+1} G_{t+1}:
//     dx = G s p,  dx_gate = G s x p (1 - p),  dz = dy h act'(z),
//     d = G (a h_{t-1} k - v kappa),  k = -w (or 1 - a: a_gate's slope of log a),  kappa = -k ds/du = k a^2 / s | k a | 0
//     da_gate = d (1 - r) (or d),  da_param = sum of d over the tokens, times sigmoid(a_param) decay / K
// The inputs are read twice: 28 bytes a value where 18 cannot be done without (bf16, gated).  8 documents, 16384 x 4096: 454 us,
// sums 157, join 13, gradients 270, da_param 8.  Issue slots (63 and 52 % taken) and the path from shared memory (51 and 62 %) bound
// it, not HBM (56 and 49 %).
struct GradParams {
    Params p;
    const void* dy;
    const float *h0, *dhT;
    void *dx, *da, *dg, *dz;
    float* dh0;
    float *P, *h, *g, *part;  // [tiles][C]
    int tiles;                // at most: T / TT + N, sequence n's from cu[n] / TT + n on
};

// A tile's first token and tokens (0: no such tile).
struct Where {
    int t0, rows;
};
template <typename T>
struct GradTile {
    static constexpr int CB = 32, VN = V16<T>::n, CH = CB / VN, NT = VN == 8 ? 128 : 256, TT = NT / CH, NQ = TT / 4;
    // CTAs an SM of the two kernels.  Smaller CTAs walk while others compute (8 documents, 16384 x 4096, bf16, when it was chosen: 483
    // us; with 256 threads and 3 and 2 CTAs 535); fewer registers spill (5 CTAs: 560).  fp32 holds half the values a thread: 267 us
    // for 16384 x 2048 so, 307 with 128 threads and 6 and 4 CTAs.
    static constexpr int SUM = VN == 8 ? 6 : 4, GRAD = VN == 8 ? 4 : 3;
    float4 a[NQ][CB], b[NQ + 1][CB], e[NQ][CB];  // units as in FwdTile; b gets the states before each token, and the last one behind them, e the G
    uint4 in[2][5][NT];                          // x, a_gate, x_gate, z, dy of this tile and the next one; then the gradients on their way to rows
    float K[2][CB];     // of this item and the next one
    Where where[2];
    float red[NT / 32][CB];
    static __device__ __forceinline__ int unit(int q, int c) { return c ^ 2 * (q & 3); }
};

// The (tile, block of channels) pairs of a CTA: blockIdx.x, + gridDim.x, ..
struct Items {
    int blocks, tile, block, tiles_on, blocks_on;
    __device__ __forceinline__ Items(int C, int CB) {
        blocks = (C + CB - 1) / CB, tile = blockIdx.x / blocks, block = blockIdx.x % blocks;
        tiles_on = gridDim.x / blocks, blocks_on = gridDim.x % blocks;
    }
    __device__ __forceinline__ Items after() const {
        Items a = *this;
        a.advance();
        return a;
    }
    __device__ __forceinline__ void advance() {
        tile += tiles_on, block += blocks_on;
        if (block >= blocks) block -= blocks, ++tile;
    }
};

// Tile v, by a warp's 32-ary search.
__device__ __forceinline__ Where tile_at(const Params& p, int TT, int v) {
    const int lane = threadIdx.x & 31;
    auto first = [&](int n) { return max(0, min(__ldg(p.cu + n), p.T)) / TT + n; };
    int lo = 0, hi = p.N;  // the last n in [lo, hi) that starts at v or before
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, n = lo + lane * step;
        const unsigned at = __ballot_sync(0xffffffffu, n < hi && first(n) <= v);
        const int k = at ? 31 - __clz((int)at) : 0;
        lo += k * step;
        hi = min(hi, lo + step);
    }
    int bos, eos;
    bounds(p.cu, lo, p.T, bos, eos);
    const int64_t off = (int64_t)(v - first(lo)) * TT;
    Where w;
    w.rows = off < 0 ? 0 : (int)max((int64_t)0, min((int64_t)TT, eos - bos - off)), w.t0 = bos + (int)(w.rows ? off : 0);
    return w;
}

// The asynchronous copies of a tile's inputs, in a group of their own; places as the workers' Share has them.  Rows behind
// the tile's end get inputs that pass everything on as it is: a = 1, no intake, no gradient of their own.
template <typename T>
__device__ __forceinline__ void copy_tile(const GradParams& q, GradTile<T>& sm, int buf, const Where& w, int c0) {
    using F = GradTile<T>;
    using Q = Share<T, F::CB>;
    const Params& p = q.p;
    const int row = threadIdx.x / F::CH, ch = threadIdx.x % F::CH, slot = Q::place(row, ch, F::CH), c = c0 + ch * F::VN;
    uint4(&to)[5][F::NT] = sm.in[buf];
    if (row >= w.rows) {
        const uint32_t inf = std::is_same<T, float>::value ? 0x7f800000u : 0x7f807f80u, open = p.ap ? inf | (inf & 0x40004000u) << 1 : inf;
        to[1][slot] = make_uint4(open, open, open, open);
        to[0][slot] = to[2][slot] = to[3][slot] = to[4][slot] = make_uint4(0u, 0u, 0u, 0u);
    } else if (c < p.C) {
        const int64_t t = w.t0 + row;
        copy16_async(&to[0][slot], static_cast<const T*>(p.x) + t * p.ldx + c);
        copy16_async(&to[1][slot], static_cast<const T*>(p.ag) + t * p.lda + c);
        if (p.xg) copy16_async(&to[2][slot], static_cast<const T*>(p.xg) + t * p.ldg + c);
        if (p.z) copy16_async(&to[3][slot], static_cast<const T*>(p.z) + t * p.ldz + c);
        copy16_async(&to[4][slot], static_cast<const T*>(q.dy) + t * p.C + c);
    }
    copy_commit();
}
// One warp finds the tile of the item after next, and works out the next item's rates, while others walk.
template <Kind KIND, typename F>
__device__ __forceinline__ void look_ahead(const GradParams& q, F& sm, int turn, int tile, int c0) {
    const Params& p = q.p;
    const int lane = threadIdx.x & 31;
    if (tile >= 0 && tile < q.tiles) {
        const Where w = tile_at(p, F::TT, tile);
        if (lane == 0) sm.where[turn] = w;
    }
    if (has_param<KIND>(p)) sm.K[turn ^ 1][lane] = c0 + lane < p.C ? rate_of(__ldg(p.ap + c0 + lane), p.decay) : 0.f;
}

// e = dy act(z) and the decays and intakes of a worker's tokens to shared memory.
template <typename T, Kind KIND>
__global__ void __launch_bounds__(GradTile<T>::NT, GradTile<T>::SUM) linrec_sum_kernel(const __grid_constant__ GradParams q) {
    using F = GradTile<T>;
    using Q = Share<T, F::CB>;
    constexpr int NP = Q::NP, CB = F::CB, NQ = F::NQ;
    extern __shared__ __align__(128) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const Params& p = q.p;
    const int lane = threadIdx.x & 31;
    const Q my(threadIdx.x);
    Items next(p.C, CB);
    Where w = tile_at(p, F::TT, next.tile);
    copy_tile(q, sm, 0, w, next.block * CB);
    if (threadIdx.x < 32) look_ahead<KIND>(q, sm, 1, next.after().tile, next.block * CB);
    for (int buf = 0; next.tile < q.tiles; buf ^= 1) {
        const int v = next.tile, c0 = next.block * CB, rows = w.rows;
        next.advance();
        copy_wait<0>();
        __syncthreads();
        if (next.tile < q.tiles) {
            w = sm.where[buf ^ 1];
            copy_tile(q, sm, buf ^ 1, w, next.block * CB);
        }
        if (!rows) {
            if (threadIdx.x / 32 == 2) look_ahead<KIND>(q, sm, buf, next.after().tile, next.block * CB);
            continue;
        }
        float2 K[NP], x[NP], ag[NP], xg[NP], a[NP], b[NP], e[NP];
        my.rates(sm.K[buf], K);
        my.load(sm.in[buf][0], x);
        my.load(sm.in[buf][1], ag);
        my.load(sm.in[buf][2], xg);
        my.load(sm.in[buf][4], e);
        steps<KIND>(p, any_far(K), K, ag, xg, x, a, b);
        if (p.z) {
            float2 z[NP];
            my.load(sm.in[buf][3], z);
            branch(p.act, z, e);
        }
        my.template put<F>(sm.a, a);
        my.template put<F>(sm.b, b);
        my.template put<F>(sm.e, e);
        __syncthreads();
        const int64_t own = (int64_t)v * p.C + c0 + lane;
        const bool ok = c0 + lane < p.C;
        if (threadIdx.x < 32) {
            float h = 0.f, P = 1.f;
#pragma unroll 4
            for (int u = 0; u < NQ; ++u) {
                const float4 av = sm.a[u][F::unit(u, lane)], bv = sm.b[u][F::unit(u, lane)];
                h = __fmaf_rn(av.x, h, bv.x), h = __fmaf_rn(av.y, h, bv.y), h = __fmaf_rn(av.z, h, bv.z), h = __fmaf_rn(av.w, h, bv.w);
                P = __fmul_rn(P, __fmul_rn(__fmul_rn(av.x, av.y), __fmul_rn(av.z, av.w)));
            }
            if (ok) q.P[own] = P, q.h[own] = h;
        } else if (threadIdx.x < 64) {
            float g = 0.f, after = 1.f;
#pragma unroll 4
            for (int u = NQ - 1; u >= 0; --u) {
                const float4 av = sm.a[u][F::unit(u, lane)], ev = sm.e[u][F::unit(u, lane)];
                g = __fmaf_rn(after, g, ev.w), g = __fmaf_rn(av.w, g, ev.z), g = __fmaf_rn(av.z, g, ev.y), g = __fmaf_rn(av.y, g, ev.x);
                after = av.x;
            }
            if (ok) q.g[own] = __fmul_rn(after, g);
        } else if (threadIdx.x < 96) {
            look_ahead<KIND>(q, sm, buf, next.after().tile, next.block * CB);
        }
    }
    copy_wait<0>();
}

// A CTA 32 channels of one sequence, in one direction (blockIdx.y): each tile's sum is replaced by what reaches the tile.  Its
// warps take an eighth of the tiles each, first from 0 and then from what the eighths before them leave.
__global__ void __launch_bounds__(256) linrec_join_kernel(const __grid_constant__ GradParams q, int TT) {
    __shared__ float Ps[8][32], vs[8][32];
    const Params& p = q.p;
    const int blocks = (p.C + 31) / 32, lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x % blocks * 32 + lane, n = blockIdx.x / blocks;
    int bos, eos;
    bounds(p.cu, n, p.T, bos, eos);
    const int tiles = (eos - bos + TT - 1) / TT, each = (tiles + 7) / 8, lo = min(warp * each, tiles), count = min(each, tiles - lo);
    const bool back = blockIdx.y, ok = c < p.C;
    const int64_t own = (int64_t)n * p.C + c, step = back ? -(int64_t)p.C : p.C;
    const int64_t at = (int64_t)(bos / TT + n + (back ? tiles - 1 - lo : lo)) * p.C + c;
    float* sum = (back ? q.g : q.h) + at;
    const float* P = q.P + at;
    constexpr int U = 8;
    float ps[U], ss[U];
    auto load = [&](int i) {  // tiles i .. of its eighth; behind its end: pass on
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool has = ok && i + k < count;
            ps[k] = has ? P[(i + k) * step] : 1.f, ss[k] = has ? sum[(i + k) * step] : 0.f;
        }
    };
    float v = 0.f, all = 1.f;
    for (int i = 0; i < count; i += U) {
        load(i);
#pragma unroll
        for (int k = 0; k < U; ++k) v = __fmaf_rn(ps[k], v, ss[k]), all = __fmul_rn(all, ps[k]);
    }
    Ps[warp][lane] = all, vs[warp][lane] = v;
    __syncthreads();
    const float* from = back ? q.dhT : q.h0;
    v = from && ok ? from[own] : 0.f;
    for (int i = 0; i < warp; ++i) v = __fmaf_rn(Ps[i][lane], v, vs[i][lane]);
    for (int i = 0; i < count; i += U) {
        if (count > U) load(i);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (ok && i + k < count) sum[(i + k) * step] = v;
            v = __fmaf_rn(ps[k], v, ss[k]);
        }
    }
    if (warp == 7 && back && q.dh0 && ok) q.dh0[own] = v;
}

template <typename T, Kind KIND>
__global__ void __launch_bounds__(GradTile<T>::NT, GradTile<T>::GRAD) linrec_bwd_kernel(const __grid_constant__ GradParams q) {
    using F = GradTile<T>;
    using Q = Share<T, F::CB>;
    constexpr int NP = Q::NP, CB = F::CB, NQ = F::NQ;
    constexpr bool bf16 = !std::is_same<T, float>::value;
    extern __shared__ __align__(128) unsigned char raw[];
    F& sm = *reinterpret_cast<F*>(raw);
    const Params& p = q.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const Q my(threadIdx.x);
    Items next(p.C, CB);  // the last tiles first: their inputs are those that the sums' kernel read last
    Where w = tile_at(p, F::TT, q.tiles - 1 - next.tile);
    copy_tile(q, sm, 0, w, next.block * CB);
    if (warp == 0) look_ahead<KIND>(q, sm, 1, q.tiles - 1 - next.after().tile, next.block * CB);
    for (int buf = 0; next.tile < q.tiles; buf ^= 1) {
        const int v = q.tiles - 1 - next.tile, c0 = next.block * CB;
        const int rows = w.rows, t0 = w.t0;
        next.advance();
        const int64_t own = (int64_t)v * p.C + c0 + lane;
        const bool ok = c0 + lane < p.C;
        float carry = 0.f;  // what reaches the tile, in the walkers
        if (rows && warp < 2 && ok) carry = warp ? q.g[own] : q.h[own];
        copy_wait<0>();
        __syncthreads();
        if (next.tile < q.tiles) {
            w = sm.where[buf ^ 1];
            copy_tile(q, sm, buf ^ 1, w, next.block * CB);
        }
        if (!rows) {
            if (q.part && threadIdx.x < CB && ok) q.part[own] = 0.f;
            if (warp == 2) look_ahead<KIND>(q, sm, buf, q.tiles - 1 - next.after().tile, next.block * CB);
            continue;
        }
        uint4(&in)[5][F::NT] = sm.in[buf];
        float2 dx[NP], dg[NP], da1[NP], da0[NP], rest[NP], dz[NP];  // factors of the gradients
        {
            float2 K[NP], x[NP], ag[NP], xg[NP], a[NP], m[NP], r[NP], k[NP], s[NP];
            my.rates(sm.K[buf], K);
            my.load(in[1], ag);
            my.load(in[0], x);
            if (has_gate<KIND>(p)) {
                my.load(in[2], xg);
                two_sigmoids(ag, xg, r, dx, rest, dg);
#pragma unroll
                for (int i = 0; i < NP; ++i) x[i] = __fmul2_rn(x[i], dx[i]);
            } else {
                one_sigmoid(ag, r, rest);
#pragma unroll
                for (int i = 0; i < NP; ++i) dx[i] = both(1.f), dg[i] = both(0.f);
            }
            if (has_param<KIND>(p)) {
                float2 w2[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i) w2[i] = __fmul2_rn(K[i], r[i]), k[i] = __fmul2_rn(w2[i], both(-1.f));
                decays(any_far(K), w2, a, m);
            } else {
                forget(r, rest, a);
#pragma unroll
                for (int i = 0; i < NP; ++i) m[i] = rest[i], k[i] = m[i], rest[i] = both(1.f);
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) da1[i] = __fmul2_rn(a[i], k[i]);
            if (scale_of<KIND>(p) == GDN_SCALE_SQRT) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float2 t = rest_of_square(a[i], m[i]);
                    const float2 o = make_float2(rsqrt_approx(fmaxf(t.x, FLT_MIN)), rsqrt_approx(fmaxf(t.y, FLT_MIN)));  // t = 0: s = 0, and k is 0 as well
                    s[i] = __fmul2_rn(t, o), da0[i] = __fmul2_rn(__fmul2_rn(da1[i], a[i]), o);
                }
            } else if (scale_of<KIND>(p) == GDN_SCALE_LINEAR) {
#pragma unroll
                for (int i = 0; i < NP; ++i) s[i] = m[i], da0[i] = da1[i];
            } else {
#pragma unroll
                for (int i = 0; i < NP; ++i) s[i] = both(1.f), da0[i] = both(0.f);
            }
            float2 b[NP], e[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                b[i] = __fmul2_rn(s[i], x[i]);
                da0[i] = __fmul2_rn(da0[i], __fmul2_rn(x[i], both(-1.f)));
                dg[i] = __fmul2_rn(b[i], dg[i]), dx[i] = __fmul2_rn(s[i], dx[i]);
            }
            my.load(in[4], e);
            if (p.z) {
                float2 z[NP];
                my.load(in[3], z);
                float2 f[NP];
                act_slope(p.act, z, f, dz);
#pragma unroll
                for (int i = 0; i < NP; ++i) dz[i] = __fmul2_rn(e[i], dz[i]), e[i] = __fmul2_rn(e[i], f[i]);
            }
            my.template put<F>(sm.a, a);
            my.template put<F>(sm.b, b);
            my.template put<F>(sm.e, e);
        }
        __syncthreads();
        if (warp == 0) {
            float h = carry;
#pragma unroll 4
            for (int j = 0; j < NQ; ++j) {
                const float4 av = sm.a[j][F::unit(j, lane)], bv = sm.b[j][F::unit(j, lane)];
                float4 o;
                o.x = h, o.y = __fmaf_rn(av.x, o.x, bv.x), o.z = __fmaf_rn(av.y, o.y, bv.y), o.w = __fmaf_rn(av.z, o.z, bv.z), h = __fmaf_rn(av.w, o.w, bv.w);
                sm.b[j][F::unit(j, lane)] = o;
            }
            sm.b[NQ][F::unit(NQ, lane)].x = h;
        } else if (warp == 1) {
            float g = carry, after = 1.f;
#pragma unroll 4
            for (int j = NQ - 1; j >= 0; --j) {
                const float4 av = sm.a[j][F::unit(j, lane)], ev = sm.e[j][F::unit(j, lane)];
                float4 o;
                o.w = __fmaf_rn(after, g, ev.w), o.z = __fmaf_rn(av.w, o.w, ev.z), o.y = __fmaf_rn(av.z, o.z, ev.y), g = o.x = __fmaf_rn(av.y, o.y, ev.x);
                after = av.x;
                sm.e[j][F::unit(j, lane)] = o;
            }
        } else if (warp == 2) {
            look_ahead<KIND>(q, sm, buf, q.tiles - 1 - next.after().tile, next.block * CB);
        }
        __syncthreads();
        float2 g[NP], old[NP], d[NP];
        my.template get<F>(sm.e, g);
        my.template get<F>(sm.b, old);
        if (p.z) {  // the state after a token is the one before the next
            float2 h[NP];
#pragma unroll
            for (int i = 0; i < NP; i += 2) {
                const float after = sm.b[my.q + 1][F::unit(my.q + 1, my.c + 4 * i)].x;  // bf16: the second channel is 8 on
                h[i] = make_float2(old[i].y, old[i + 1].x), h[i + 1] = make_float2(old[i + 1].y, after);
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) dz[i] = __fmul2_rn(dz[i], h[i]);
        }
        float2 total[NP / 2];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            d[i] = __fmul2_rn(g[i], __ffma2_rn(da1[i], old[i], da0[i]));
            dx[i] = __fmul2_rn(g[i], dx[i]), dg[i] = __fmul2_rn(g[i], dg[i]);
        }
        if (q.part) {
#pragma unroll
            for (int i = 0; i < NP; i += 2) total[i / 2] = __fadd2_rn(d[i], d[i + 1]);
            if constexpr (bf16) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float t = __fadd_rn(total[i].x, total[i].y);
                    t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    if (lane % 4 == 0) sm.red[my.q / 4][my.c + 8 * i] = t;
                }
            } else {
                sm.red[warp][lane] = __fadd_rn(total[0].x, total[0].y);
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) d[i] = __fmul2_rn(d[i], rest[i]);
        if constexpr (bf16) {  // through the inputs' places to whole rows: with a warp's 32 bytes a row, 16 rows a store, the stores took most of the path to memory
            my.put_in(in[0], dx);
            my.put_in(in[1], d);
            if (has_gate<KIND>(p)) my.put_in(in[2], dg);
            if (p.z) my.put_in(in[3], dz);
            __syncthreads();
            const int row = threadIdx.x / F::CH, ch = threadIdx.x % F::CH, slot = Q::place(row, ch, F::CH), c = c0 + ch * F::VN;
            if (row < rows && c < p.C) {
                const int64_t to = (int64_t)(t0 + row) * p.C + c;
                st16_stream(static_cast<T*>(q.dx) + to, in[0][slot]);
                st16_stream(static_cast<T*>(q.da) + to, in[1][slot]);
                if (has_gate<KIND>(p)) st16_stream(static_cast<T*>(q.dg) + to, in[2][slot]);
                if (p.z) st16_stream(static_cast<T*>(q.dz) + to, in[3][slot]);
            }
        } else {
            const int64_t to = (int64_t)(t0 + 4 * my.q) * p.C + c0 + my.c;
            auto out = [&](void* y, const float2 (&o)[NP]) {
                const float f[4] = {o[0].x, o[0].y, o[1].x, o[1].y};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * my.q + j < rows) __stcs(static_cast<float*>(y) + to + (int64_t)j * p.C, f[j]);
            };
            if (c0 + my.c < p.C) {
                out(q.dx, dx);
                out(q.da, d);
                if (has_gate<KIND>(p)) out(q.dg, dg);
                if (p.z) out(q.dz, dz);
            }
            if (q.part) __syncthreads();
        }
        if (q.part && threadIdx.x < CB && ok) {
            float t = sm.red[0][lane];
#pragma unroll
            for (int i = 1; i < (bf16 ? F::TT / 16 : F::NT / 32); ++i) t = __fadd_rn(t, sm.red[i][lane]);
            q.part[own] = t;
        }
    }
    copy_wait<0>();
}

// da_param: a CTA 32 channels; its warps add the tiles' sums warp, warp + 8, .., then the warps' in order.
__global__ void __launch_bounds__(256) linrec_param_kernel(int tiles, int C, float decay, const float* __restrict__ ap,
                                                           const float* __restrict__ part, float* __restrict__ out) {
    __shared__ float sums[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x / 32;
    float s = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int i = warp; i < tiles; i += 8) s = __fadd_rn(s, __ldg(part + (int64_t)i * C + c));
    }
    sums[warp][threadIdx.x & 31] = s;
    __syncthreads();
    if (warp || c >= C) return;
    for (int i = 1; i < 8; ++i) s = __fadd_rn(s, sums[i][threadIdx.x]);
    const float v = __ldg(ap + c), K = rate_of(v, decay), sp = 1.f / (1.f + expf(-v));
    out[c] = K == 0.f ? 0.f : s * (decay * sp / K);  // (NaN where a_param is)
}

template <typename T, typename F>
Params strides(Params q) {
    constexpr int64_t tile = (int64_t)F::TT * sizeof(T);
    q.sx = tile * q.ldx, q.sa = tile * q.lda, q.sg = tile * q.ldg, q.sz = tile * q.ldz, q.sy = tile * q.C;
    return q;
}
template <typename T, int CB, int WORKERS, int CTAS>
gdn_status launch_fwd_of(cudaStream_t s, const Params& p) {
    using F = FwdTile<T, CB, WORKERS>;
    const Kind kind = kind_of(p);
    auto* kernel = kind == kBothGates ? linrec_fwd_kernel<T, F, CB, CTAS, kBothGates> : kind == kForget ? linrec_fwd_kernel<T, F, CB, CTAS, kForget> : linrec_fwd_kernel<T, F, CB, CTAS, kAny>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess) return GDN_ERR_CUDA;
    const unsigned ctas = (unsigned)((p.C + CB - 1) / CB) * (unsigned)p.N;
    Params q = strides<T, F>(p);
    q.ranked = p.N > 1 && p.N <= kRanked && ctas > (unsigned)(kSMs * CTAS) && (long long)p.N * p.N * p.N <= 256LL * p.T;
    kernel<<<ctas, F::NT, sizeof(F), s>>>(q);
    return launch_status();
}
// Short sequences by themselves, in a second launch what is left: worth it where the CTAs that it saves are many.  us so and with a CTA each,
// bf16, gated: 256 sequences of 1 token x 4096 13.5, 244; 4096 of 1 104, 3892; 1024 of 4 on average 58, 1121; 256 of 16 65, 301, of 32 173, 319,
// of 64 335, 362, of 128 479, 461; 16 of 1 x 8192 3.6, 35, of 56 65, 54.  fp32 the same way: 256 of 1 13.8, 217, of 32 185, 307, of 64 353, 378, of 128 564, 549.
template <typename T, int CB, int WORKERS, int CTAS>
gdn_status launch_many(cudaStream_t s, const Params& p) {
    const long long cut = (p.C / V16<T>::n + 127) / 128;
    linrec_short_kernel<T><<<(unsigned)(cut * p.N), 128, 0, s>>>(p);
    gdn_status st = launch_status();
    if (st != GDN_OK || p.T <= kShort) return st;
    using F = FwdTile<T, CB, WORKERS>;
    const Kind kind = kind_of(p);
    auto* kernel = kind == kBothGates ? linrec_long_kernel<T, F, CB, CTAS, kBothGates> : kind == kForget ? linrec_long_kernel<T, F, CB, CTAS, kForget> : linrec_long_kernel<T, F, CB, CTAS, kAny>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess) return GDN_ERR_CUDA;
    const int blocks = (p.C + CB - 1) / CB, most = 4 * CTAS * kSMs / blocks, groups = most < 1 ? 1 : most < p.N ? most : p.N;
    kernel<<<(unsigned)blocks * (unsigned)groups, F::NT, sizeof(F), s>>>(strides<T, F>(p), groups);
    return launch_status();
}
// Which form, by the number n of CTAs of 32 channels.  A token takes a CTA, bf16 and gated, 7 ns with 16 channels and 512 workers, 10 ns
// with 32 and 512, 12 ns with 32 and 256, and 19 ns each of two of the last kind on one SM; a batch of several sequences ends with its
// longest alone, which 16 channels shorten where the lengths differ and do not where they are near one another (the host does not
// know them).  us with the three forms, bf16 / fp32:
//     1 x 16384 x 1024 (n = 32)             113, 160, 200 / 121, 189, 263
//     1 x 16384 x 4096 (128)                230, 161, 202 / 238, 210, 280
//     2 of 13142 and 2858 x 2048 (128)      111, 132, 165 / 122, 158, 216
//     2 of 4882 and 3118 x 2048 (128)        64,  52,  63 /  66,  64,  86
//     3 ragged, 16000 x 1600 (150)           87,  95, 118 /  97, 119, 158
//     2, 8000 x 2560 (160)                   83,  69,  77 /  90,  86,  95
//     4, 8192 x 2048 (256)                   65,  50,  65 /  68,  63,  79
//     1 x 16384 x 8192 (256)                459, 318, 305 / 489, 436, 407
//     13, 20000 x 2560 (1040)               184, 125, 108 / 193, 167, 154
//     16, 32768 x 4096 (2048)               451, 307, 265 / 472, 416, 398
// launch_many goes by the mean length alone: 255 sequences of one token beside one of 65536 x 2048 are past it and take 806 us, the long
// one alone 444 (with a branch; one of 8192 x 4096 168 and 86).
template <typename T>
gdn_status launch_fwd(cudaStream_t s, const Params& p) {
    const long long n = (long long)((p.C + 31) / 32) * p.N;
    if (n > 2 * kSMs && p.T < (n > 64 * kSMs ? 128LL : 48LL) * p.N) return launch_many<T, 32, 256, 2>(s, p);
    if (n <= kSMs / 2 || (p.N > 1 && n <= kSMs)) return launch_fwd_of<T, 16, 512, 1>(s, p);
    if (n <= kSMs + kSMs / 8 || (p.N >= 4 && n <= 2 * kSMs + kSMs / 8)) return launch_fwd_of<T, 32, 512, 1>(s, p);
    return launch_fwd_of<T, 32, 256, 2>(s, p);
}

int64_t grad_tiles(int T, int N, int dtype) { return (int64_t)T / (dtype == GDN_BF16 ? GradTile<__nv_bfloat16>::TT : GradTile<float>::TT) + N; }

template <typename T>
gdn_status launch_bwd(cudaStream_t s, const GradParams& q) {
    using F = GradTile<T>;
    const Params& p = q.p;
    const Kind kind = kind_of(p);
    auto* sum = kind == kBothGates ? linrec_sum_kernel<T, kBothGates> : kind == kForget ? linrec_sum_kernel<T, kForget> : linrec_sum_kernel<T, kAny>;
    auto* bwd = kind == kBothGates ? linrec_bwd_kernel<T, kBothGates> : kind == kForget ? linrec_bwd_kernel<T, kForget> : linrec_bwd_kernel<T, kAny>;
    if (cudaFuncSetAttribute(sum, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess ||
        cudaFuncSetAttribute(bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(F)) != cudaSuccess)
        return GDN_ERR_CUDA;
    const int64_t items = (int64_t)q.tiles * ((p.C + F::CB - 1) / F::CB);
    auto ctas = [&](int each) { return (unsigned)(items < kSMs * each ? items : kSMs * each); };
    if (p.T > 0) {
        sum<<<ctas(F::SUM), F::NT, sizeof(F), s>>>(q);
        const gdn_status st = launch_status();
        if (st != GDN_OK) return st;
    }
    linrec_join_kernel<<<dim3((unsigned)((p.C + 31) / 32) * (unsigned)p.N, 2), 256, 0, s>>>(q, F::TT);
    gdn_status st = launch_status();
    if (st != GDN_OK || p.T == 0) return st;
    bwd<<<ctas(F::GRAD), F::NT, sizeof(F), s>>>(q);
    return launch_status();
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
    // CTAs are numbered, states per sequence, channels up to the end of a block and tokens a few tiles behind the last indexed in 31 bits
    if (s->T_total > INT_MAX - 4096 || s->C > INT_MAX - 64 || (long long)s->N * s->C >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
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
    // Rows a thread: bf16, of which registers hold 5 CTAs an SM, as many as make it one wave, up to 8; fp32 up to 3.  us with 1, 2, 3, 6, 8 rows,
    // gated, bf16: 128 x 4096 3.8, 3.8, 4.6, 5.9, 7.4; 256 x 4096 7.3, 6.4, 7.4, 10.3, 12.0; 512 x 8192 18.6, 17.8, 17.4, 16.9, 18.1; 2048 x 8192 60.0, 54.5, 53.4,
    // 52.9, 52.9; fp32: 256 x 2560 4.6, 5.1, 5.8, 8.2, 9.8; 512 x 4096 12.0, 11.6, 11.2, 13.1, 14.1; 2048 x 8192 70.3, 68.3, 68.3, 68.7, 69.0.
    const bool bf16 = shape->dtype == GDN_BF16;
    const int blocks = (p.C / (bf16 ? 8 : 4) + 127) / 128, wave = kSMs * (bf16 ? 5 : 12), most = bf16 ? 8 : 3;
    const long long want = ((long long)blocks * p.N + wave - 1) / wave;
    const int rows = (int)(want < most ? want : most);
    const unsigned grid = (unsigned)blocks * (unsigned)((p.N + rows - 1) / rows);
    if (shape->dtype == GDN_BF16) linrec_update_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p, rows);
    else linrec_update_kernel<float><<<grid, 128, 0, s>>>(p, rows);
    return launch_status();
}

extern "C" size_t gdn_linear_recurrence_bwd_workspace_size(const gdn_linrec_shape* shape) {
    using namespace gdn;
    if (check_linrec(shape, false, false, false) != GDN_OK) return 0;
    return 4 * (size_t)grad_tiles(shape->T_total, shape->N, shape->dtype) * shape->C * sizeof(float);
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
    q.dh0 = d_init_state;
    q.tiles = (int)grad_tiles(p.T, p.N, shape->dtype);
    const size_t each = (size_t)q.tiles * p.C;
    q.P = static_cast<float*>(workspace), q.h = q.P + each, q.g = q.h + each, q.part = da_param ? q.g + each : nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.N > 0) {
        st = shape->dtype == GDN_BF16 ? launch_bwd<__nv_bfloat16>(s, q) : launch_bwd<float>(s, q);
        if (st != GDN_OK) return st;
    }
    if (!da_param) return GDN_OK;
    linrec_param_kernel<<<(unsigned)((p.C + 31) / 32), 256, 0, s>>>(p.T > 0 ? q.tiles : 0, p.C, p.decay, a_param, q.part, da_param);
    return launch_status();
}
