/*
 * seq.h -- C ABI of the sequence operators in libdgrad_gb300.so, on one NVIDIA
 * GB300 (sm_103a): what a selective state-space layer runs between its matrix
 * products, forwards, backwards and for single tokens.
 *
 *   seq_conv   the short causal depthwise convolution (and its gradients)
 *   seq_scan   the selective state-space scan
 *   seq_norm   the norms around a block with its gate and residual scale
 *
 * Tensors are token-major: channels are innermost and contiguous, a token's
 * and a batch row's distance are given in elements (seq_ref_t), so that a
 * slice of a wider projection is read or written in place.  Activations are
 * fp32, fp16 or bf16 (one type for all of a plan's activations); states of
 * the scan, parameters and the parameters' gradients are fp32.  All sums,
 * states and statistics are held in fp32; a 16-bit output is rounded once.
 *
 * Ownership, errors and streams follow dgrad.h: the caller owns the tensors;
 * a plan owns its device workspace and is bound to the device that was
 * current when it was made; one plan must not run on two streams at once (its
 * workspace is shared); streams are passed as void * holding a cudaStream_t.
 * The first backward call of a plan allocates its share of the workspace (so
 * make one before capturing a graph); nothing else allocates.  A plan's
 * batch, length and rows are the largest that its calls may bring; each call
 * gives its own.  The workspace is sized for the largest, by cudaMalloc, and
 * kept until the plan is destroyed; seq_*_workspace_bytes() says how much that
 * is without (gradients 0) and with backward calls (1), and each operator's
 * part below what it grows with.  Where there is no room the call returns
 * DGRAD_ERR_OOM, has launched nothing and can be made again.  Outputs are fully overwritten; an output that overlaps an
 * input returns DGRAD_ERR_ALIAS (interleaved slices of one buffer do not
 * overlap), a pointer that is not a multiple of its element size
 * DGRAD_ERR_MISALIGNED (16-byte alignment and strides are faster, and not
 * needed), a missing tensor DGRAD_ERR_INVALID_ARG.  Results do not depend on
 * timing: no sum uses atomics.
 *
 * Limits: a call has at least one batch row and token (or row); a row may be
 * empty by its length.  Distances (seq_ref_t) are not negative, those of tokens
 * and groups below 2^28; batch rows may lie any distance apart.  seq_conv: K
 * 2 to 4.  seq_scan: up to 128 states, channels * states within 31 bits.
 * seq_norm: up to 8192 channels.  Larger sizes
 * return DGRAD_ERR_UNSUPPORTED when the plan is made.
 *
 * Rows of unequal length: `lengths` (int32, one per batch row, device memory,
 * may be NULL: all full) says how many leading tokens of each row are there;
 * values outside [0, length] are taken as the nearest bound.  What lies behind
 * is never read, outputs and gradients there are 0, and states stop at the
 * last token (a row of length 0 hands its state on unchanged).
 *
 * An infinity or NaN within a row reaches what the formulas below give it to,
 * in its row and channel (of B or C: group), and nothing else.
 */
#ifndef SEQ_GB300_H
#define SEQ_GB300_H

#include <stddef.h>

#include "dgrad.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { SEQ_F32 = 0, SEQ_F16 = 1, SEQ_BF16 = 2 } seq_dtype_t;
typedef enum { SEQ_ACT_NONE = 0, SEQ_ACT_SILU = 1, SEQ_ACT_SIGMOID = 2 } seq_act_t;

/* A strided tensor: elements from one batch row, token and group to the next;
 * channels (states of B and C) are contiguous.  ptr NULL: absent. */
typedef struct {
    void *ptr;
    long long sb, st, sg;
} seq_ref_t;

/* ------------------------------------------------------------------ seq_conv
 *   pre[b,t,d] = bias[d] + sum over k < K of weight[d,k] * x[b, t-K+1+k, d]
 *   y = act(pre), act the identity or SiLU
 * with x before the first token taken from `state` ([batch, K-1, channels],
 * oldest first, contiguous; NULL: zeros).  final_state receives the last K-1
 * inputs of each row (earlier state rows among them where the row is shorter).
 * K is 2, 3 or 4.  Workspace with gradients: 4 (K + 1) channels P bytes, P the
 * larger of batch ceil(length / 256) and 768 SMs / ceil(channels / 4) + 1 + batch. */
typedef struct seq_conv_plan_s *seq_conv_plan_t;

typedef struct {
    long long batch, length;
    seq_ref_t x, y;
    const float *weight;   /* [channels, K] */
    const float *bias;     /* [channels] or NULL */
    const int *lengths;
    const void *state;
    void *final_state;
} seq_conv_args_t;

typedef struct {
    long long batch, length;
    seq_ref_t grad_y, x, grad_x;
    const float *weight, *bias;
    const int *lengths;
    const void *state, *grad_final;   /* grad_final: gradient of final_state, NULL: none */
    void *grad_state;                 /* NULL: not wanted; needs state */
    float *grad_weight, *grad_bias;   /* grad_bias NULL: not wanted */
} seq_conv_grad_args_t;

/* One token of `batch` sequences: x, y [batch, channels] (sb is the row
 * distance).  cache [n_slots, K-1, channels], contiguous; row i reads slot
 * slots[i] and writes slot write_slots[i] (NULL: slots; slots NULL: i).  A row
 * whose slot to read is negative is padding: its y is 0 and no state changes;
 * a negative slot to write keeps the cache as it is.  Slots at or beyond
 * n_slots are refused by the kernel the same way and recorded
 * (seq_conv_check returns DGRAD_ERR_INVALID_ARG).  A slot that one row writes
 * must not be read or written by another row of the same call. */
typedef struct {
    long long batch, n_slots;
    seq_ref_t x, y;
    const float *weight, *bias;
    void *cache;
    const int *slots, *write_slots;
} seq_conv_step_args_t;

dgrad_status_t seq_conv_plan(long long batch, long long length, long long channels, int width, seq_dtype_t dtype,
                             seq_act_t act, seq_conv_plan_t *plan_out);
dgrad_status_t seq_conv_run(seq_conv_plan_t plan, const seq_conv_args_t *args, void *stream);
dgrad_status_t seq_conv_backward(seq_conv_plan_t plan, const seq_conv_grad_args_t *args, void *stream);
dgrad_status_t seq_conv_step(seq_conv_plan_t plan, const seq_conv_step_args_t *args, void *stream);
dgrad_status_t seq_conv_check(seq_conv_plan_t plan);
size_t seq_conv_workspace_bytes(seq_conv_plan_t plan, int gradients);
void seq_conv_destroy(seq_conv_plan_t plan);

/* ------------------------------------------------------------------ seq_scan
 *   delta = softplus(dt + dt_bias)
 *   h_t[d,n] = exp(delta_t[d] A[d,n]) h_(t-1)[d,n] + delta_t[d] u_t[d] B_t[g,n]
 *   y_t[d] = sum over n of C_t[g,n] h_t[d,n] + D[d] u_t[d]
 *   out = y * SiLU(z)
 * with A <= 0 in any real use, channel d in group g = d / (channels / groups).
 * D, dt_bias, z may be absent.  state and final_state: [batch, channels,
 * states] fp32, contiguous (state NULL: zeros).
 *
 * checkpoints (training): seq_scan_checkpoint_bytes() bytes that the run
 * fills with the states at every 8th token and the backward call reads.
 *
 * Workspace, with C = min(64, length / 16) chunks and P the channels, each
 * group's rounded up to a multiple of 4: 4 batch C P (states + 1) bytes (none
 * where C is 1 or less).  Gradients add 4 batch C P (states + 2) and, for the
 * parts of grad_B and grad_C, 32 q T batch length groups bytes: q is states / 4
 * rounded up to a power of two, T the column tiles of a group, of 256, 128, 128,
 * 64, 32, 16 channels for q = 1, 2, 4, 8, 16, 32.  Those parts grow with states
 * times channels: 1 KB a token and group at 16 states and 1024 channels, 131 KB
 * at 64 states and 8192 channels, 524 KB at 128. */
typedef struct seq_scan_plan_s *seq_scan_plan_t;

typedef struct {
    long long batch, length;
    seq_ref_t u, dt, B, C, z, out;
    const float *A;         /* [channels, states] */
    const float *D, *dt_bias; /* [channels] or NULL */
    const int *lengths;
    const float *state;
    float *final_state;
    float *checkpoints;     /* NULL: not wanted */
} seq_scan_args_t;

typedef struct {
    long long batch, length;
    seq_ref_t grad_out, u, dt, B, C, z;
    seq_ref_t grad_u, grad_dt, grad_B, grad_C, grad_z;   /* grad_z present exactly if z is */
    const float *A, *D, *dt_bias;
    const int *lengths;
    const float *state, *checkpoints, *grad_final;
    float *grad_state;                       /* NULL: not wanted */
    float *grad_A, *grad_D, *grad_dt_bias;   /* grad_D, grad_dt_bias NULL: not wanted */
} seq_scan_grad_args_t;

/* One token of `batch` sequences; cache [n_slots, channels, states] fp32, slots
 * as in seq_conv_step_args_t.  u, dt, z, out [batch, channels]; B, C [batch,
 * groups, states]. */
typedef struct {
    long long batch, n_slots;
    seq_ref_t u, dt, B, C, z, out;
    const float *A, *D, *dt_bias;
    float *cache;
    const int *slots, *write_slots;
} seq_scan_step_args_t;

dgrad_status_t seq_scan_plan(long long batch, long long length, long long channels, int states, int groups,
                             seq_dtype_t dtype, seq_scan_plan_t *plan_out);
size_t seq_scan_checkpoint_bytes(seq_scan_plan_t plan, long long batch, long long length);
dgrad_status_t seq_scan_run(seq_scan_plan_t plan, const seq_scan_args_t *args, void *stream);
dgrad_status_t seq_scan_backward(seq_scan_plan_t plan, const seq_scan_grad_args_t *args, void *stream);
dgrad_status_t seq_scan_step(seq_scan_plan_t plan, const seq_scan_step_args_t *args, void *stream);
dgrad_status_t seq_scan_check(seq_scan_plan_t plan);
size_t seq_scan_workspace_bytes(seq_scan_plan_t plan, int gradients);
void seq_scan_destroy(seq_scan_plan_t plan);

/* ------------------------------------------------------------------ seq_norm
 *   p = y * rsqrt(mean(y^2) + eps) * post_weight   (post_weight NULL: p = y)
 *   b = act(gate) * p                              (gate absent: b = p)
 *   r' = residual + scale * b                      (scale NULL: 1)
 *   x = r' * rsqrt(mean(r'^2) + eps) * next_weight
 * over rows of `channels`: the norm after a block, its gate and per-channel
 * residual scale, the residual add and the norm before the next block.  r' is
 * stored in the residual's type (the activations' or fp32); x is formed from
 * the unrounded r'.  sb is the row distance of each tensor.  The backward call
 * recomputes what it needs from the forward's inputs.  Workspace with gradients:
 * 12 channels bytes for each block (at most 10 an SM). */
typedef struct seq_norm_plan_s *seq_norm_plan_t;

typedef struct {
    long long rows;
    seq_ref_t y, gate, residual, residual_out, x;
    const float *post_weight, *scale, *next_weight;
} seq_norm_args_t;

typedef struct {
    long long rows;
    seq_ref_t y, gate, residual, grad_residual_out, grad_x;   /* grad_residual_out absent: zeros */
    seq_ref_t grad_y, grad_gate, grad_residual;
    const float *post_weight, *scale, *next_weight;
    float *grad_post_weight, *grad_scale, *grad_next_weight;  /* present exactly if the parameter is */
} seq_norm_grad_args_t;

dgrad_status_t seq_norm_plan(long long rows, long long channels, seq_dtype_t dtype, seq_dtype_t residual_dtype,
                             seq_act_t gate_act, float eps, seq_norm_plan_t *plan_out);
dgrad_status_t seq_norm_run(seq_norm_plan_t plan, const seq_norm_args_t *args, void *stream);
dgrad_status_t seq_norm_backward(seq_norm_plan_t plan, const seq_norm_grad_args_t *args, void *stream);
size_t seq_norm_workspace_bytes(seq_norm_plan_t plan, int gradients);
void seq_norm_destroy(seq_norm_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* SEQ_GB300_H */
