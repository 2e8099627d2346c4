/*
 * gdn_layer.h -- C ABI of the Gated DeltaNet layer's ops either side of the
 * recurrence (sm_103a): the gate activations that turn the layer's raw
 * projections into (g, beta), the short causal depthwise convolution over the
 * q/k/v projections with its per-sequence conv state cache (prefill and
 * decode, and its gradient), the norm of the queries' and keys' heads with
 * the position rotation in the same pass (and its gradient), and the gated
 * RMSNorm applied to the recurrence's output.
 *
 * "Defending Against the Training-Inference Numeric Mismatch in RL
 * (Especially Linear Attention)" keeps these ops identical on the trainer and
 * the generator (section 3.1: one model definition, with A_log kept in fp32
 * through the trainer's bf16 wrapping) and reuses the serving engine's conv
 * state cache unchanged (section 3.2).  Their formulas are the standard GDN
 * layer's:
 *
 *     g    = -exp(A_log[h]) * softplus(a + dt_bias[h]),   beta = sigmoid(b)
 *     conv y[t, c] = act( bias[c] + sum_{i<W} w[c, i] * xw[t + i, c] ),
 *          xw = (the W-1 rows before the sequence: its conv state) ++ (its rows)
 *     norm y = o / sqrt(mean(o^2) + eps) * weight * silu(z)   (per row of d)
 *     q/k  n = x * r * weight,  r = 1 / sqrt(sum(x^2) * c + eps),  c = 1/d (RMS) or 1 (L2),
 *          then the pairs (u, v) of n's first rotary_dim values by the token's angles:
 *          (u cos - v sin, v cos + u sin)
 *
 * Invariance.  Every output element is computed by one thread with one fixed
 * order of operations that depends on nothing but its own row (conv: its own
 * sequence's rows): results do not depend on the batch, on how a batch is
 * tiled, or on whether a token goes through the prefill or the decode entry
 * point (gdn_causal_conv1d_fwd and gdn_causal_conv1d_update share the
 * per-element arithmetic, so prefill-then-update is bit-identical to one
 * prefill over the whole sequence).
 *
 * Memory and ownership as in gdn.h: caller-owned, dense row-major DEVICE
 * pointers; x, y, o, z, the conv state, the conv weight and the RMSNorm
 * weight 16-byte aligned; g, beta, A_log, dt_bias, the conv bias, cu_seqlens,
 * state_indices and has_initial_state 4-byte aligned (a and b: their element
 * size).  Misalignment returns GDN_ERR_INVALID_ARG.  Nothing is allocated;
 * every call is one asynchronous launch on `stream` (a cudaStream_t; NULL =
 * legacy default stream) and returns host-side validation or launch errors
 * only (the two gradients are two launches each and take a workspace).
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gate activations.  a, b: [T, HV] in in_dtype (bf16 or fp32, the projection
 * outputs); A_log, dt_bias: [HV] fp32 (dt_bias may be NULL: zero).  Writes
 * g = -exp(A_log) * softplus(a + dt_bias) and beta = sigmoid(b), both [T, HV]
 * fp32, the inputs gdn_recurrent_fwd / gdn_decode_step take.  softplus(x) is
 * log(1 + exp(x)), taken as x itself above x = 20.
 */
gdn_status gdn_gates(int64_t T, int HV, gdn_dtype in_dtype, const void* a, const void* b,
                     const float* A_log, const float* dt_bias, float* g, float* beta,
                     void* stream);

/*
 * Gated RMSNorm over the last axis: o, z, y are [rows, d] in dtype (for the
 * recurrence's output rows = T * HV and d = dv); weight [d] fp32.  z may be
 * NULL (no gate: plain RMSNorm).  y may alias o.  d must be a multiple of 8
 * (bf16) or 4 (fp32) and at most 2048; eps >= 0.  The sum of squares of a row
 * is taken in fp32 in one fixed order (each lane of a fixed lane group sums
 * its own 16-byte chunks in ascending order, then a fixed xor butterfly).
 */
gdn_status gdn_gated_rmsnorm(int64_t rows, int d, gdn_dtype dtype, const void* o, const void* z,
                             const float* weight, float eps, void* y, void* stream);

typedef struct {
    int N;           /* sequences (update: batch size) */
    int T_total;     /* packed tokens (update: must equal N) */
    int C;           /* channels, e.g. q, k and v projections side by side */
    int W;           /* taps, 2..8 */
    gdn_dtype dtype; /* x, y and the conv state */
    int activation;  /* 1: SiLU on the output; 0: none */
} gdn_conv_shape;

/*
 * Causal depthwise conv over a packed varlen batch (prefill, trainer forward).
 * x, y [T_total, C]; weight [C, W] fp32 (tap W-1 multiplies the current row);
 * bias [C] fp32 or NULL; cu_seqlens int32 [N + 1] as in gdn.h.  conv_state is
 * a pool [num_slots, W-1, C] in dtype (NULL: every sequence starts from zeros
 * and no state is written); sequence n uses slot state_indices[n]
 * (state_indices NULL: slot n, and num_slots must be >= N).  The slot's rows
 * are read as the sequence's initial state when has_initial_state is NULL or
 * has_initial_state[n] != 0 (else zeros), and are then overwritten with the
 * sequence's final state, the last W-1 rows of (initial state ++ its rows); a
 * sequence of length 0 leaves its slot as it was (or zeroes it when its
 * initial state is off).  A negative or out-of-range slot: zero initial
 * state, nothing written.  Slots of different sequences must differ; y must
 * not alias x.  C must be a multiple of 8 (bf16) or 4 (fp32).
 */
gdn_status gdn_causal_conv1d_fwd(const gdn_conv_shape* shape, const void* x, const float* weight,
                                 const float* bias, const int32_t* cu_seqlens, void* conv_state,
                                 const int32_t* state_indices, int num_slots,
                                 const int32_t* has_initial_state, void* y, void* stream);

/*
 * One decode token per sequence: x, y [N, C] (shape->T_total == N); the
 * pool conv_state [num_slots, W-1, C] is updated in place (rows shift up by
 * one, x enters as the newest row).  Sequence b uses slot state_indices[b]
 * (NULL: slot b, and num_slots must be >= N); a negative or out-of-range slot
 * skips it (y row untouched).  Slots of different sequences must differ; y
 * must not alias x.  Bit-identical to running gdn_causal_conv1d_fwd one
 * token further.
 */
gdn_status gdn_causal_conv1d_update(const gdn_conv_shape* shape, const void* x, const float* weight,
                                    const float* bias, void* conv_state,
                                    const int32_t* state_indices, int num_slots, void* y,
                                    void* stream);

/*
 * Gradient of gdn_causal_conv1d_fwd for the loss L = sum <d_y, y> +
 * <d_final_state, final state>.  x, weight, bias (NULL: zero), cu_seqlens as
 * given to the forward; init_state [N, W-1, C] in dtype is the initial state
 * of each sequence, in the order of the sequences (NULL: zeros).  d_y
 * [T_total, C]; d_final_state [N, W-1, C] in dtype (NULL: zero).  Writes dx
 * [T_total, C] in dtype, dweight [C, W] and dbias [C] fp32 (dbias NULL: not
 * written) and d_init_state [N, W-1, C] in dtype (NULL: not written).  Rows of
 * dx that no sequence covers are left as they are.  The outputs must not alias
 * the inputs.  fp32 sums; each sum's order is fixed by the shape and
 * cu_seqlens, so results are deterministic; dweight and dbias are not
 * batch-invariant.  d_y, dx, d_final_state and d_init_state 16-byte aligned,
 * dweight and dbias 4-byte aligned.
 */
size_t gdn_causal_conv1d_bwd_workspace_size(const gdn_conv_shape* shape);

gdn_status gdn_causal_conv1d_bwd(const gdn_conv_shape* shape, const void* x, const float* weight,
                                 const float* bias, const int32_t* cu_seqlens,
                                 const void* init_state, const void* d_y,
                                 const void* d_final_state, void* dx, float* dweight, float* dbias,
                                 void* d_init_state, void* workspace, size_t workspace_bytes,
                                 void* stream);

typedef enum { GDN_NORM_RMS = 0, GDN_NORM_L2 = 1 } gdn_norm;

typedef struct {
    int64_t T;         /* tokens */
    int HQ, HK;        /* heads of q and of k (any numbers; HK = 0: no k) */
    int d;             /* head dim, a multiple of 8 (bf16) or 4 (fp32), at most 256 */
    int rotary_dim;    /* leading values of a head that are rotated, a multiple of 16 (bf16) or 8 (fp32); 0: none */
    int interleaved;   /* pairs: 0: (i, i + rotary_dim/2); 1: (2i, 2i + 1) */
    int norm;          /* gdn_norm */
    int max_positions; /* rows of cos and sin */
    float eps;
    gdn_dtype dtype;   /* q, k, their outputs and gradients */
    int64_t ldq, ldk;  /* elements from one token's q (k) to the next one's: at least HQ * d (HK * d) */
} gdn_qk_shape;

/*
 * Norm of each head of q [T, HQ, d] and k [T, HK, d] and rotation by the
 * token's position, in one pass.  The heads of a token are dense; tokens are
 * ldq (ldk) elements apart, so q and k may be columns of one wider row, such
 * as the conv's output.  q_weight, k_weight [d] fp32 or NULL (ones).  cos, sin
 * [max_positions, rotary_dim / 2] fp32; token t uses row positions[t] (int32;
 * positions NULL: row t, and max_positions must be >= T).  A token whose
 * position is negative or not below max_positions is skipped: its rows of the
 * outputs are left as they are (with rotary_dim = 0, positions is not read and no token
 * is skipped).  Outputs q_out [T, HQ, d], k_out [T, HK, d] dense in dtype; they
 * may alias q and k where those are dense.  Each row is computed by one lane
 * group in one fixed order: results do not depend on T or the other rows.
 * Strides are multiples of 8 (bf16) or 4 (fp32) elements.  q, k, the outputs, the
 * weights, cos and sin are 16-byte aligned, positions 4-byte aligned.
 */
gdn_status gdn_qk_norm_rope(const gdn_qk_shape* shape, const void* q, const void* k,
                            const float* q_weight, const float* k_weight, const float* cos,
                            const float* sin, const int32_t* positions, void* q_out, void* k_out,
                            void* stream);

/*
 * Its gradient: from q, k (the inputs) and d_q_out, d_k_out (dense), dq and dk
 * with lddq (lddk) elements from token to token, and, where the weight is
 * given, dq_weight and dk_weight [d] fp32 (NULL: not written).  dq may alias
 * d_q_out and dk may alias d_k_out where they are dense; a skipped token's rows
 * are left as they are and add nothing to the weights' gradients.  fp32 sums in
 * an order fixed by the shape.
 */
size_t gdn_qk_norm_rope_bwd_workspace_size(const gdn_qk_shape* shape);

gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_shape* shape, const void* q, const void* k,
                                const float* q_weight, const float* k_weight, const float* cos,
                                const float* sin, const int32_t* positions, const void* d_q_out,
                                const void* d_k_out, void* dq, void* dk, int64_t lddq, int64_t lddk,
                                float* dq_weight, float* dk_weight, void* workspace,
                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H_ */
