/*
 * gdn_linrec.h -- C ABI of the gated linear recurrence (sm_103a): one state per
 * channel, a decay per token and channel, behind the short causal conv of
 * gdn_layer.h and on the same kind of slots as the selective scan of
 * gdn_scan.h.  Prompts and trainer forward, single tokens on a pool of
 * states, and the gradient.
 *
 * For every sequence (tokens cu_seqlens[n] .. cu_seqlens[n+1]-1 of a packed
 * batch) and channel c of C:
 *
 *     r_t = sigmoid(a_gate[t, c])
 *     a_t = exp(-decay softplus(a_param[c]) r_t)   (a_param NULL: a_t = r_t)
 *     s_t = sqrt(1 - a_t^2)  or  1 - a_t  or  1     (scale)
 *     h_t = a_t h_{t-1} + s_t x[t, c] sigmoid(x_gate[t, c])
 *     y_t = h_t act(z[t, c])
 *
 * x_gate NULL: x is taken as it is; z NULL: y = h.  act is silu(z) = z
 * sigmoid(z) or gelu(z) = z sigmoid(2 sqrt(2 / pi) (z + 0.044715 z^3)) (the
 * tanh form).  1 - a is taken as -expm1 of the exponent and 1 - a^2 as
 * (1 - a)(1 + a), so that decays next to 1 keep their inputs' scale (1 - a
 * below 2^-126 counts as 0; decay softplus(a_param) past 3e38 counts as 3e38).  An
 * a_gate of -inf under an a_param keeps the state and takes nothing in (scale
 * sqrt and linear); without an a_param it forgets the state, and +inf keeps it
 * bit for bit (scale one adds the input all the same).  A decay is never above 1.
 *
 * The factor s_t holds for every token, a sequence's first too.  For a layer that
 * takes the first token's input unscaled, the state after that token is its
 * x sigmoid(x_gate) and its y that state's: give it as the initial state and
 * start from the second token (d_init_state is then its gradient).
 *
 * Invariance.  The bits of y and of the final state of a sequence depend only
 * on that sequence's own inputs: not on the batch around it, and not on
 * whether its tokens arrive in one gdn_linear_recurrence_fwd call, in several
 * chained through the state, or one by one through
 * gdn_linear_recurrence_update.  A channel's tokens are walked in order, one
 * fused multiply-add each, and nothing is split over time.
 *
 * Memory and ownership as in gdn.h: caller-owned DEVICE pointers.  x, a_gate,
 * x_gate, z, y [T_total, C] in dtype; a_param [C] and every state [.., C] fp32.
 * The inputs x, a_gate, x_gate, z have row strides in the shape, so they may
 * be columns of wider rows (a projection's output); everything else is dense.
 * x, a_gate, x_gate, z, y, d_y, dx, da_gate, dx_gate, dz, a_param, da_param, every state and the
 * workspace 16-byte aligned, the rest 4-byte aligned; strides multiples of 16 bytes; C a
 * multiple of 8 (bf16) or 4 (fp32).  Tokens that no sequence covers (behind
 * cu_seqlens[N]) are not read, and their rows of the outputs are left as they
 * are.  Calls are asynchronous on `stream`, allocate nothing and return
 * host-side validation or launch errors only.
 */
#ifndef GDN_LINREC_H_
#define GDN_LINREC_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GDN_SCALE_SQRT = 0, GDN_SCALE_LINEAR = 1, GDN_SCALE_ONE = 2 } gdn_input_scale;
typedef enum { GDN_ACT_SILU = 0, GDN_ACT_GELU = 1 } gdn_act;

typedef struct {
    int N;           /* sequences (update: batch size) */
    int T_total;     /* packed tokens (update: must equal N) */
    int C;           /* channels */
    gdn_dtype dtype; /* x, a_gate, x_gate, z, y and their gradients */
    int scale;       /* gdn_input_scale */
    int activation;  /* gdn_act, of z */
    float decay;     /* > 0 and finite; with a_param only */
    int64_t ldx, lda, ldg, ldz; /* elements from one token's row to the next one's: x, a_gate, x_gate, z */
} gdn_linrec_shape;

/*
 * The recurrence over a packed varlen batch.  state is a pool [num_slots, C]
 * (NULL: every sequence starts from zeros and no state is written); sequence n
 * uses slot state_indices[n] (state_indices NULL: slot n, and num_slots must
 * be >= N).  The slot is read as the sequence's initial state when
 * has_initial_state is NULL or has_initial_state[n] != 0 (else zeros), and is
 * then overwritten with the final state; a sequence of length 0 leaves its
 * slot as it was (or zeroes it when its initial state is off).  A negative or
 * out-of-range slot: zero initial state, nothing written.  Slots of different
 * sequences must differ; y must not alias an input.  cu_seqlens as in gdn.h,
 * except that cu_seqlens[N] may be below T_total.
 */
gdn_status gdn_linear_recurrence_fwd(const gdn_linrec_shape* shape, const void* x, const void* a_gate,
                                     const float* a_param, const void* x_gate, const void* z,
                                     const int32_t* cu_seqlens, float* state,
                                     const int32_t* state_indices, int num_slots,
                                     const int32_t* has_initial_state, void* y, void* stream);

/*
 * One token per sequence (shape->T_total == N): the slots of the pool are
 * updated in place, y [N, C].  A negative or out-of-range slot skips its row
 * (y row untouched).  The slots in use must differ.  One launch, no
 * workspace: capturable as it is.
 */
gdn_status gdn_linear_recurrence_update(const gdn_linrec_shape* shape, const void* x, const void* a_gate,
                                        const float* a_param, const void* x_gate, const void* z,
                                        float* state, const int32_t* state_indices, int num_slots,
                                        void* y, void* stream);

/*
 * Gradient for the loss L = sum <d_y, y> + <d_final_state, final state>.
 * init_state, d_final_state [N, C] fp32, in the order of the sequences (NULL:
 * zeros).  Writes dx, da_gate, dx_gate, dz [T_total, C] in dtype (dense;
 * dx_gate and dz required when x_gate and z are given, else ignored),
 * da_param [C] fp32 (NULL: not written) and d_init_state [N, C] fp32 (NULL:
 * not written).  Outputs must not alias inputs.  The states are recomputed;
 * nothing of the forward call is needed.  fp32 sums, each in an order fixed by
 * the shape and cu_seqlens: deterministic; the sum over tokens in da_param is
 * not batch-invariant.  (Where 1 - a_t is 0, the slope of scale sqrt is
 * infinite and a_gate's share of the exponent 0; their product is taken as 0.)
 *
 * The workspace holds four fp32 values per channel and tile of 32 tokens, at
 * most T_total / 32 + N tiles: half a byte per token and channel, and 16 C bytes
 * per sequence, empty ones too.
 */
size_t gdn_linear_recurrence_bwd_workspace_size(const gdn_linrec_shape* shape);

gdn_status gdn_linear_recurrence_bwd(const gdn_linrec_shape* shape, const void* x, const void* a_gate,
                                     const float* a_param, const void* x_gate, const void* z,
                                     const int32_t* cu_seqlens, const float* init_state,
                                     const void* d_y, const float* d_final_state, void* dx,
                                     void* da_gate, float* da_param, void* dx_gate, void* dz,
                                     float* d_init_state, void* workspace, size_t workspace_bytes,
                                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINREC_H_ */
