/*
 * gdn_scan.h -- C ABI of the selective state space scan (sm_103a): the other
 * linear recurrence that hybrid models put behind the short causal conv of
 * gdn_layer.h.  Prompts and trainer forward, single tokens on a pool of
 * states, and the gradient.
 *
 * For every sequence (tokens cu_seqlens[n] .. cu_seqlens[n+1]-1 of a packed
 * batch), channel c of C, state s of S, with group g = c / (C / G):
 *
 *     d_t      = softplus(dt[t, c] + dt_bias[c])     (dt_softplus != 0, else dt + dt_bias)
 *     h_t[c,s] = exp(-d_t exp(A_log[c, s])) h_{t-1}[c,s] + d_t x[t, c] B[t, g, s]
 *     y[t, c]  = (sum_s h_t[c,s] Cm[t, g, s] + D[c] x[t, c]) * silu(z[t, c])
 *
 * D NULL: no skip term; z NULL: no gate; dt_bias NULL: zero.
 *
 * Invariance.  The bits of y and of the final state of a sequence depend only
 * on that sequence's own inputs: not on the batch around it, and not on
 * whether its tokens arrive in one gdn_selective_scan_fwd call, in several
 * chained through the state, or one by one through
 * gdn_selective_scan_update.  A channel's tokens are walked in order, its
 * states summed in one fixed tree, and nothing is split over time.
 *
 * Memory and ownership as in gdn.h: caller-owned DEVICE pointers.  x, dt, z, y
 * [T_total, C] and B, Cm [T_total, G, S] in dtype; A_log [C, S], D, dt_bias [C]
 * and every state [.., C, S] fp32.  The inputs x, dt, z, B, Cm have row
 * strides in the shape, so they may be columns of wider rows (a projection's
 * output); everything else is dense.  x, dt, z, B, Cm, y, d_y, dx, ddt, dz, dB, dC, A_log,
 * every state and the workspace 16-byte aligned, the rest 4-byte aligned; strides multiples of 16
 * bytes.  Supported: S in {8, 16, 32, 64}; C / G a multiple of 8.  Tokens that
 * no sequence covers (behind cu_seqlens[N]) are not read, and their rows of the
 * outputs are left as they are.  Calls are asynchronous on `stream`, allocate
 * nothing and return host-side validation or launch errors only.
 */
#ifndef GDN_SCAN_H_
#define GDN_SCAN_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int N;           /* sequences (update: batch size) */
    int T_total;     /* packed tokens (update: must equal N) */
    int C;           /* channels */
    int G;           /* groups of channels that share B and Cm, C % G == 0 */
    int S;           /* states per channel: 8, 16, 32 or 64 */
    gdn_dtype dtype; /* x, dt, z, B, Cm, y and their gradients */
    int dt_softplus;
    int64_t ldx, lddt, ldz, ldB, ldC; /* elements from one token's row to the next one's */
} gdn_scan_shape;

/*
 * Scan over a packed varlen batch.  state is a pool [num_slots, C, S] (NULL:
 * every sequence starts from zeros and no state is written); sequence n uses
 * slot state_indices[n] (state_indices NULL: slot n, and num_slots must be >=
 * N).  The slot is read as the sequence's initial state when has_initial_state
 * is NULL or has_initial_state[n] != 0 (else zeros), and is then overwritten
 * with the final state; a sequence of length 0 leaves its slot as it was (or
 * zeroes it when its initial state is off).  A negative or out-of-range slot:
 * zero initial state, nothing written.  Slots of different sequences must
 * differ; y must not alias an input.  cu_seqlens as in gdn.h, except that
 * cu_seqlens[N] may be below T_total.
 */
gdn_status gdn_selective_scan_fwd(const gdn_scan_shape* shape, const void* x, const void* dt,
                                  const float* A_log, const void* B, const void* Cm,
                                  const float* D, const void* z, const float* dt_bias,
                                  const int32_t* cu_seqlens, float* state,
                                  const int32_t* state_indices, int num_slots,
                                  const int32_t* has_initial_state, void* y, void* stream);

/*
 * One token per sequence (shape->T_total == N): the slots of the pool are
 * updated in place, y [N, C].  A negative or out-of-range slot skips its row
 * (y row untouched).  The slots in use must differ.  One launch, no
 * workspace: capturable as it is.
 */
gdn_status gdn_selective_scan_update(const gdn_scan_shape* shape, const void* x, const void* dt,
                                     const float* A_log, const void* B, const void* Cm,
                                     const float* D, const void* z, const float* dt_bias,
                                     float* state, const int32_t* state_indices, int num_slots,
                                     void* y, void* stream);

/*
 * Gradient for the loss L = sum <d_y, y> + <d_final_state, final state>.
 * init_state, d_final_state [N, C, S] fp32, in the order of the sequences (NULL: zeros).
 * Writes dx, ddt, dz [T_total, C] and dB, dC [T_total, G, S] in dtype (dense;
 * dz required when z is given, else ignored), dA_log [C, S], dD, ddt_bias [C]
 * fp32 (dD and ddt_bias NULL: not written) and d_init_state [N, C, S] fp32
 * (NULL: not written).  Outputs must not alias inputs.  The states are
 * recomputed; nothing of the forward call is needed.  fp32 sums, each in an order fixed
 * by the shape and cu_seqlens: deterministic, but the sums over tokens and
 * channels are not batch-invariant.
 *
 * The workspace is large: per channel and state it holds an fp32 value every 8 tokens and two per
 * segment, that is 16 to 128 tokens of a sequence (at most T_total / 16 + N segments), and
 * 8 S bytes per token and block of 64 (S 32 and 64: 32) channels of a group.  For few
 * sequences that is 6 bytes for every byte of a bf16 x at 16 states (12 for small batches, whose
 * segments are shorter), 27 at 64; every further sequence, empty ones too, adds 8 C S bytes, as much
 * as its init_state and d_init_state together.
 */
size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_shape* shape);

gdn_status gdn_selective_scan_bwd(const gdn_scan_shape* shape, const void* x, const void* dt,
                                  const float* A_log, const void* B, const void* Cm,
                                  const float* D, const void* z, const float* dt_bias,
                                  const int32_t* cu_seqlens, const float* init_state,
                                  const void* d_y, const float* d_final_state, void* dx, void* ddt,
                                  float* dA_log, void* dB, void* dC, float* dD, void* dz,
                                  float* ddt_bias, float* d_init_state, void* workspace,
                                  size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SCAN_H_ */
